"""Measured cases of the 8-bit paged cache and of rotary positions with several axes: new keys and values quantised as
they are written into a paged cache, the cache read back as packed 16-bit rows, the attention of new tokens over it, and
the per-head norm with a rotation whose angles come from several positions a token (time, height, width), with its
gradient.

A cached row of one head is E4M3 codes times one power of two, 2^(scale byte - 127): the smallest that brings the row's
largest magnitude to at most 448, within the limits that keep every value exact in the row's 16-bit type.

`run` computes the operators in their plain form (elementary torch operations, 32 bits, rounded once), or, where `own` is
true, through this package's entry points. `exact` computes the same from the definitions in 64 bits.
"""
import math

import numpy as np
import torch

if __name__ == "__main__":
    raise SystemExit("a module of cases; import it")

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
LIMITS = {"bf16": (-80, 80), "fp16": (-15, 7)}  # exponents of a row's scale
EPS = 1e-6
THETA = 10000.0
WORKSPACE_BYTES = 256 << 20  # scratch that a serving program keeps for its attention calls


# ------------------------------------------------------------------------------------------------ cases
def axes_case(name, kind, tokens, hq, hkv, d, sections, pairs, dtype, fused, max_pos):
    """sections: pairs of each axis, in order, as text; pairs: "half" (i, i + rot/2) or "adjacent" (2i, 2i+1);
    fused: q and k are slices of one projection's output rows."""
    return dict(name=name, kind=kind, tokens=tokens, hq=hq, hkv=hkv, d=d, sections=sections, pairs=pairs, dtype=dtype,
                fused=fused, max_pos=max_pos)


def cache_case(name, kind, batch, q_lo, q_hi, kv_lo, kv_hi, hq, hkv, d, dv, page, order, dtype, window=-1, causal=True, pad=0,
               sections=""):
    """A batch whose new tokens (read8: keys read back) number q_lo..q_hi and whose total lengths, those among them,
    kv_lo..kv_hi, evenly spaced; order: "nhd" pages hold [slot][head][d], "hnd" [head][slot][d]; window: keys left of
    the diagonal, -1 all; pad: rows behind the last sequence; append8: sections norm q and k and rotate them on the way."""
    return dict(name=name, kind=kind, batch=batch, q_lo=q_lo, q_hi=q_hi, kv_lo=kv_lo, kv_hi=kv_hi, hq=hq, hkv=hkv, d=d, dv=dv,
                page=page, order=order, dtype=dtype, window=window, causal=causal, pad=pad, sections=sections)


def listed():
    return [
        # one decode step of a few sequences of a model of text and images: latency
        axes_case("axes_step", "axes", 4, 32, 8, 128, "16,24,24", "half", "bf16", True, 8192),
        # a prompt's or training step's tokens, straight from the fused projection
        axes_case("axes_train", "axes", 18000, 32, 8, 128, "16,24,24", "half", "bf16", True, 8192),
        # frames of a video: adjacent pairs, sections that no vector width divides, every head its own keys
        axes_case("axes_bwd_video", "axes_bwd", 4099, 16, 16, 128, "22,21,21", "adjacent", "fp16", False, 8192),
        # the gradient for a training step's tokens, half of a 256-wide head rotated
        axes_case("axes_bwd_train", "axes_bwd", 18000, 16, 8, 256, "24,20,20", "half", "bf16", True, 8192),
        # decode: every sequence appends one token, normed, rotated and quantised on the way
        cache_case("append8_step", "append8", 33, 1, 1, 1, 1000, 32, 8, 128, 128, 16, "nhd", "bf16", sections="16,24,24"),
        # prefill chunks of uneven length quantised into pages of another head order
        cache_case("append8_chunk_d256", "append8", 7, 1, 4001, 9, 6007, 16, 8, 256, 256, 64, "hnd", "bf16"),
        # the last keys of a sliding-window layer's sequences read back for their next chunks
        cache_case("read8_window_d256", "read8", 13, 1, 1025, 1, 8192, 16, 8, 256, 256, 64, "hnd", "fp16"),
        # whole contexts of a batch of prompts read back
        cache_case("read8_prompts", "read8", 8, 2000, 16384, 2000, 16384, 32, 8, 128, 128, 16, "nhd", "bf16", pad=5),
        # one user's next token over a short context: latency
        cache_case("decode8_one", "paged8", 1, 1, 1, 999, 999, 32, 8, 128, 128, 16, "nhd", "bf16"),
        # a serving batch of uneven contexts, one token each
        cache_case("decode8_batch", "paged8", 64, 1, 1, 500, 16384, 32, 8, 128, 128, 16, "nhd", "bf16", pad=3),
        # sliding-window layer of the same kind of batch
        cache_case("decode8_window_d256", "paged8", 48, 1, 1, 1, 8192, 16, 8, 256, 256, 64, "hnd", "fp16", window=1024),
        # wide query/key heads with narrower value heads, a few speculative tokens each, all keys seen
        cache_case("spec8_d192", "paged8", 9, 0, 5, 5, 4097, 32, 8, 192, 128, 48, "nhd", "bf16", causal=False),
    ]


def spread(rng, lo, hi):
    """A whole number of [lo, hi], its logarithm uniform."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def cut(rng, pairs):
    """`pairs` pairs divided between two to four axes, as text."""
    n = rng.choice([2, 3, 3, 3, 4])
    step = rng.choice([1, 4, 4])
    at = sorted(rng.sample(range(1, pairs // step), n - 1))
    return ",".join(str(step * (b - a)) for a, b in zip([0] + at, at + [pairs // step]))


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        most[c["kind"]] = {x: max(most.get(c["kind"], {}).get(x, 0), w[x]) for x in ("bytes", "flops")}
    while True:
        kind = rng.choice(["axes", "axes_bwd", "append8", "read8", "paged8", "paged8"])
        d = rng.choice([128, 128, 128, 256, 512, 192])
        hq, hkv = rng.choice([(32, 8), (16, 8), (16, 4), (16, 16), (8, 1), (14, 2), (10, 10), (32, 1)])
        dtype = rng.choice(["bf16", "fp16"])
        sections = cut(rng, rng.choice([d, d, d // 2, 64]) // 2)
        if kind in ("axes", "axes_bwd"):
            c = axes_case("", kind, spread(rng, 1, 18000), hq, hkv, d, sections, rng.choice(["half", "adjacent"]), dtype,
                          rng.random() < 0.5, 8192)
        else:
            q_hi = rng.choice([1, 1, spread(rng, 2, 16), spread(rng, 16, 64 if kind == "paged8" else 4096)])
            kv_hi = spread(rng, max(q_hi, 8), 16384)
            if kind == "read8":
                q_hi = rng.choice([q_hi, kv_hi])
            c = cache_case("", kind, spread(rng, 1, 100), rng.choice([min(1, q_hi), 0, q_hi]), q_hi,
                           max(1, int(kv_hi * rng.random())), kv_hi, hq, hkv, d, 128 if d == 192 else d,
                           rng.choice([16, 32, 64, 128, 256, 48]), rng.choice(["nhd", "hnd"]), dtype,
                           rng.choice([-1, -1, spread(rng, 1, 4096)]) if kind == "paged8" else -1,
                           kind != "paged8" or rng.random() < 0.8, rng.choice([0, 0, spread(rng, 1, 100)]),
                           rng.choice(["", sections]) if kind == "append8" else "")
            if not c["causal"]:
                c["window"] = -1
            elems = c["batch"] * kv_hi * max(hkv * d, hq * q_hi if kind == "paged8" else 0)
            if elems > 1.2e9 or sum(q for q, _ in lengths(c)) == 0:  # the plain form pads every sequence to the longest
                continue
        w = work(c)
        if all(w[x] <= most[kind][x] for x in w):
            del c["name"]
            return c


def lengths(c):
    """(new tokens, total length) of every sequence, before the seed shuffles their order."""
    n = c["batch"]
    at = [i / (n - 1) if n > 1 else 1.0 for i in range(n)]
    total = [c["kv_lo"] + round((c["kv_hi"] - c["kv_lo"]) * f) for f in at]
    new = [c["q_lo"] + round((c["q_hi"] - c["q_lo"]) * f) for f in at]
    if c["kind"] == "read8":
        return [(min(q, k), k) for q, k in zip(new, total)]
    order = sorted(range(n), key=lambda i: (i * 7919) % n if math.gcd(7919, n) == 1 else i)
    return [(new[i], max(new[i], k)) for i, k in zip(order, total)]


def rotated(c):
    """Values of a head that turn."""
    return 2 * sum(int(x) for x in c["sections"].split(",")) if c["sections"] else 0


def work(c):
    axes = len(c["sections"].split(",")) if c["sections"] else 0
    if c["kind"] in ("axes", "axes_bwd"):
        rows, heads, fwd = c["tokens"], c["hq"] + c["hkv"], c["kind"] == "axes"
        extra = rows * (4 * rotated(c) + 4 * axes) + (2 if fwd else 2 + 4) * 2 * c["d"]
        return {"bytes": (2 if fwd else 3) * 2 * rows * heads * c["d"] + extra, "flops": (8 if fwd else 18) * rows * heads * c["d"]}
    seqs = lengths(c)
    new = sum(q for q, _ in seqs)
    row = c["hkv"] * (c["d"] + c["dv"])  # values of a token's K and V
    if c["kind"] == "append8":
        q_row = c["hq"] * c["d"] if axes else 0
        return {"bytes": new * (3 * row + 2 * c["hkv"] + 4 * q_row + 4 + 4 * rotated(c) + 4 * axes) + 8 * c["batch"],
                "flops": 3 * new * row + (8 * new * (c["hq"] + c["hkv"]) * c["d"] if axes else 0)}
    if c["kind"] == "read8":
        return {"bytes": new * (3 * row + 2 * c["hkv"]) + 4 * sum(-(-q // c["page"]) for q, _ in seqs) + 8 * c["batch"],
                "flops": new * row}
    kv_rows, pairs = 0, 0
    for q, k in seqs:
        if q == 0:
            continue
        if not c["causal"]:
            kv_rows, pairs = kv_rows + k, pairs + q * k
            continue
        first = 0 if c["window"] < 0 else max(0, k - q - c["window"])
        kv_rows += k - first
        top = np.arange(k - q + 1, k + 1, dtype=np.int64)
        pairs += int(np.sum(top if c["window"] < 0 else np.minimum(top, c["window"] + 1)))
    return {"bytes": kv_rows * (row + 2 * c["hkv"]) + new * c["hq"] * (2 * c["d"] + 2 * c["dv"] + 4)
            + 4 * sum(-(-k // c["page"]) for q, k in seqs if q) + 8 * c["batch"],
            "flops": 2 * pairs * c["hq"] * (c["d"] + c["dv"])}


# ------------------------------------------------------------------------------------------------ inputs
def table(max_pos, rot):
    """[max_pos, rot] float32: rot/2 cosines, then rot/2 sines of position * THETA^(-2i/rot)."""
    freq = THETA ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    angle = torch.arange(max_pos, dtype=torch.float64, device=DEV)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], dim=1).float()


def normal(gen, shape, dtype, mean=0.0, std=1.0):
    return (torch.randn(shape, device=DEV, generator=gen) * std + mean).to(dtype)


def projected(gen, rows, c, widths):
    """Rows of heads as a projection leaves them: slices of one buffer, or a buffer each."""
    dt = DTYPES[c["dtype"]]
    if c.get("fused", True):
        whole, at, out = normal(gen, (rows, sum(h * d for h, d in widths)), dt), 0, []
        for h, d in widths:
            out.append(whole[:, at:at + h * d].unflatten(1, (h, d)))
            at += h * d
        return out
    return [normal(gen, (rows, h, d), dt) for h, d in widths]


def axis_positions(rng, tokens, axes, max_pos):
    """int32 [axes, tokens]: a running position, and patches' places in frames of up to 64 rows and columns around it."""
    base = np.arange(tokens) % (max_pos - 64)
    return torch.from_numpy(np.stack([base + (rng.integers(0, 64, tokens) if a else 0) for a in range(axes)]).astype(np.int32)).to(DEV)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV).manual_seed(seed * 2 + 1)
    rng = np.random.default_rng(seed)
    dt, d = DTYPES[c["dtype"]], c["d"]
    s = {"case": c, "sections": tuple(int(x) for x in c["sections"].split(",")) if c["sections"] else None}
    if c["sections"]:
        s["q_weight"], s["k_weight"] = normal(gen, (d,), dt, 1.0, 0.2), normal(gen, (d,), dt, 1.0, 0.2)
    if c["kind"] in ("axes", "axes_bwd"):
        s["q"], s["k"] = projected(gen, c["tokens"], c, [(c["hq"], d), (c["hkv"], d)])
        s["cos_sin"] = table(c["max_pos"], rotated(c))
        s["positions"] = axis_positions(rng, c["tokens"], len(s["sections"]), c["max_pos"])
        if c["kind"] == "axes_bwd":
            s["dq_out"] = normal(gen, (c["tokens"], c["hq"], d), dt)
            s["dk_out"] = normal(gen, (c["tokens"], c["hkv"], d), dt)
        return s
    seqs = lengths(c)
    seqs = [seqs[i] for i in rng.permutation(len(seqs))]
    new, total = np.array([q for q, _ in seqs]), np.array([k for _, k in seqs])
    rows = int(new.sum()) + c["pad"]
    cols = -(-int(total.max()) // c["page"])
    pages = int(sum(-(-total // c["page"]))) + 5
    ids = rng.permutation(pages)
    tab, at = np.full((c["batch"], cols), -1, np.int32), 0  # -1 behind a sequence's last page
    for b, k in enumerate(total):
        n = -(-int(k) // c["page"])
        tab[b, :n] = ids[at:at + n]
        at += n
    s["block_table"] = torch.from_numpy(tab).to(DEV)
    s["kv_lens"] = torch.from_numpy(total.astype(np.int32)).to(DEV)
    s["cu_seqlens_q"] = torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).to(DEV)
    s["max_seqlen_q"], s["max_seqlen_kv"] = c["q_hi"], max(c["kv_hi"], c["q_hi"])
    heads = (pages, c["page"], c["hkv"]) if c["order"] == "nhd" else (pages, c["hkv"], c["page"])
    for x, w in (("k", d), ("v", c["dv"])):
        size = torch.randn(heads, device=DEV, generator=gen).mul_(0.5).exp_()  # a token's magnitude
        s[x + "_cache"], s[x + "_scale"] = quantised(torch.randn(heads + (w,), device=DEV, generator=gen) * size[..., None], c)
    if c["kind"] == "append8":
        s["q"], s["k"], s["v"] = projected(gen, rows, c, [(c["hq"], d), (c["hkv"], d), (c["hkv"], c["dv"])])
        if c["sections"]:
            s["cos_sin"] = table(c["kv_hi"] + 64, rotated(c))
            s["positions"] = axis_positions(rng, rows, len(s["sections"]), c["kv_hi"] + 64)
            s["q_out"] = torch.zeros((rows, c["hq"], d), dtype=dt, device=DEV)
    elif c["kind"] == "read8":
        s["k_out"] = torch.zeros((rows, c["hkv"], d), dtype=dt, device=DEV)
        s["v_out"] = torch.zeros((rows, c["hkv"], c["dv"]), dtype=dt, device=DEV)
    else:
        s["q"] = normal(gen, (rows, c["hq"], d), dt)
        s["out"] = torch.zeros((rows, c["hq"], c["dv"]), dtype=dt, device=DEV)
        s["lse"] = torch.zeros((rows, c["hq"]), device=DEV)
        s["workspace"] = torch.empty(WORKSPACE_BYTES, dtype=torch.uint8, device=DEV)
        s["scale"] = d ** -0.5
    return s


# ------------------------------------------------------------------------------------------------ plain forms
def quantised(x, c):
    """The codes and the scale bytes of rows x (32 bits)."""
    lo, hi = LIMITS[c["dtype"]]
    top = x.abs().amax(-1)
    m, e = torch.frexp(top)  # top = m 2^e, m in [0.5, 1): the scale is 2^(e - 9), twice that from 448 = 0.875 2^9 on
    e = torch.where(top == 0, lo, (e - 9 + (m > 0.875).int()).clamp(lo, hi))
    codes = torch.ldexp(x, -e[..., None]).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8), (e + 127).to(torch.uint8)


def values(codes, scale):
    """What codes and scale bytes stand for, in 32 bits."""
    return torch.ldexp(codes.view(torch.float8_e4m3fn).float(), scale.int()[..., None] - 127)


def axis_angles(s):
    """[tokens, rot] cosines and sines: each pair's from the position on its own axis."""
    sections, half = s["sections"], sum(s["sections"])
    axis = torch.repeat_interleave(torch.arange(len(sections), device=DEV), torch.tensor(sections, device=DEV), output_size=half)
    pair = torch.arange(half, device=DEV)
    at = s["positions"].long()[axis].T  # [tokens, pairs]
    return torch.cat([s["cos_sin"][at, pair], s["cos_sin"][at, half + pair]], dim=1)


def rotate(x, cos_sin, pairs, back=False):
    """x [rows, heads, d] with its leading values rotated by their row's angles (backwards: by the negative)."""
    rot = cos_sin.shape[1]
    cos, sin = cos_sin[:, None, :rot // 2], cos_sin[:, None, rot // 2:]
    sin = -sin if back else sin
    head, tail = x[..., :rot], x[..., rot:]
    if pairs == "half":
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        head = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    else:
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    return torch.cat([head, tail], dim=-1)


def norm(x, weight, cos_sin, pairs):
    x = x.float()
    r = 1.0 / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)
    return rotate(x * r * weight.float(), cos_sin, pairs)


def norm_back(dy, x, weight, cos_sin, pairs):
    x = x.float()
    r = 1.0 / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)
    g, xr = rotate(dy.float(), cos_sin, pairs, back=True), x * r
    gw = g * weight.float()
    dx = r * (gw - xr * (gw * xr).mean(-1, keepdim=True))
    return dx, (g * xr).sum((0, 1), dtype=torch.float64).float()


def places(s, rows):
    """Sequence, position and liveness of every row of the batch."""
    cu, at = s["cu_seqlens_q"].long(), torch.arange(rows, device=DEV)
    seq = torch.clamp((at[:, None] >= cu[None, 1:]).sum(1), max=cu.numel() - 2)
    new = cu[seq + 1] - cu[seq]
    return seq, s["kv_lens"].long()[seq] - new + (at - cu[seq]), at < cu[-1]


def run_append(s, c):
    rows = s["k"].shape[0]
    seq, pos, live = places(s, rows)
    k, v = s["k"].float(), s["v"].float()
    if c["sections"]:
        angles = axis_angles(s)
        k = norm(s["k"], s["k_weight"], angles, "half")
        s["q_out"][live] = norm(s["q"], s["q_weight"], angles, "half").to(s["q_out"].dtype)[live]
    seq, pos = seq[live], pos[live]
    ids, slot = s["block_table"].long()[seq, pos // c["page"]], pos % c["page"]
    for name, x in (("k", k), ("v", v)):
        for cache, put in zip((s[name + "_cache"], s[name + "_scale"]), quantised(x[live], c)):
            (cache if c["order"] == "nhd" else cache.transpose(1, 2))[ids, slot] = put
    return append_outputs(s, c)


def append_outputs(s, c):
    """The updated caches as the values that their bytes stand for: E4M3 codes, and powers of two."""
    out = [s["k_cache"].view(torch.float8_e4m3fn), s["k_scale"].view(torch.float8_e8m0fnu),
           s["v_cache"].view(torch.float8_e4m3fn), s["v_scale"].view(torch.float8_e8m0fnu)]
    return out + ([s["q_out"]] if c["sections"] else [])


def run_read(s, c):
    seq, pos, live = places(s, s["k_out"].shape[0])
    seq, pos = seq[live], pos[live]
    ids, slot = s["block_table"].long()[seq, pos // c["page"]], pos % c["page"]
    for x in ("k", "v"):
        codes, scale = s[x + "_cache"], s[x + "_scale"]
        if c["order"] == "hnd":
            codes, scale = codes.transpose(1, 2), scale.transpose(1, 2)
        s[x + "_out"][live] = values(codes[ids, slot], scale[ids, slot]).to(s[x + "_out"].dtype)
    return s["k_out"], s["v_out"]


def run_paged(s, c):
    cu, lens = s["cu_seqlens_q"].long(), s["kv_lens"].long()
    hq, hkv, page = c["hq"], c["hkv"], c["page"]
    key = torch.arange(s["max_seqlen_kv"], device=DEV)
    ids = s["block_table"].long().clamp(min=0)[:, key // page]
    there = key[None, :] < lens[:, None]                                              # [batch, keys]

    def gather(x):                                                                    # [batch, hkv, keys, width]
        codes, scale = s[x + "_cache"], s[x + "_scale"]
        if c["order"] == "hnd":
            codes, scale = codes.transpose(1, 2), scale.transpose(1, 2)
        return (values(codes[ids, key % page], scale[ids, key % page]) * there[:, :, None, None]).transpose(1, 2)

    i = torch.arange(s["max_seqlen_q"], device=DEV)
    new = cu[1:] - cu[:-1]
    row = (cu[:-1, None] + i[None, :]).clamp(max=max(s["q"].shape[0] - 1, 0))
    live = i[None, :] < new[:, None]                                                  # [batch, queries]
    q = s["q"][row].float().unflatten(2, (hkv, hq // hkv)).permute(0, 2, 3, 1, 4)      # [batch, hkv, group, queries, d]
    score = torch.matmul(q.flatten(2, 3), gather("k").transpose(2, 3)).unflatten(2, (hq // hkv, -1)) * s["scale"]
    seen = there[:, None, :] & live[:, :, None]
    if c["causal"]:
        pos = (lens - new)[:, None] + i[None, :]
        seen = seen & (key[None, None, :] <= pos[:, :, None])
        if c["window"] >= 0:
            seen = seen & (key[None, None, :] >= pos[:, :, None] - c["window"])
    score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), gather("v")).unflatten(2, (hq // hkv, -1))
    o = o / torch.where(total == 0, torch.ones_like(total), total)
    lse = (top + torch.log(total)).squeeze(-1)
    s["out"][row[live]] = o.permute(0, 3, 1, 2, 4).flatten(2, 3)[live].to(s["out"].dtype)
    s["lse"][row[live]] = lse.permute(0, 3, 1, 2).flatten(2, 3)[live]
    return s["out"], s["lse"]


def run(state):
    s, c = state, state["case"]
    if own:
        return run_own(s, c)
    if c["kind"] == "axes":
        angles, dt = axis_angles(s), s["q"].dtype
        return (norm(s["q"], s["q_weight"], angles, c["pairs"]).to(dt), norm(s["k"], s["k_weight"], angles, c["pairs"]).to(dt))
    if c["kind"] == "axes_bwd":
        angles, dt = axis_angles(s), s["q"].dtype
        dq, dwq = norm_back(s["dq_out"], s["q"], s["q_weight"], angles, c["pairs"])
        dk, dwk = norm_back(s["dk_out"], s["k"], s["k_weight"], angles, c["pairs"])
        return dq.to(dt), dk.to(dt), dwq, dwk
    return {"append8": run_append, "read8": run_read, "paged8": run_paged}[c["kind"]](s, c)


def run_own(s, c):
    import scaled_dot_product_02_gb300 as sdpa

    if c["kind"] == "axes":
        return sdpa.sdpa_qk_norm_rope(s["q"], s["k"], s["q_weight"], s["k_weight"], s["cos_sin"], s["positions"], eps=EPS,
                                      interleaved=c["pairs"] == "adjacent", sections=s["sections"])
    if c["kind"] == "axes_bwd":
        return sdpa.sdpa_qk_norm_rope_bwd(s["dq_out"], s["dk_out"], s["q"], s["k"], s["q_weight"], s["k_weight"], s["cos_sin"],
                                          s["positions"], eps=EPS, interleaved=c["pairs"] == "adjacent", sections=s["sections"])
    cache = (s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["block_table"], s["kv_lens"], s["cu_seqlens_q"])
    if c["kind"] == "append8":
        if c["sections"]:
            sdpa.sdpa_paged_append_fp8(s["k"], s["v"], *cache, cache_layout=c["order"], q=s["q"], q_weight=s["q_weight"],
                                       k_weight=s["k_weight"], cos_sin=s["cos_sin"], positions=s["positions"],
                                       sections=s["sections"], eps=EPS, q_out=s["q_out"])
        else:
            sdpa.sdpa_paged_append_fp8(s["k"], s["v"], *cache, cache_layout=c["order"])
        return append_outputs(s, c)
    if c["kind"] == "read8":
        return sdpa.sdpa_paged_read_fp8(*cache, cache_layout=c["order"], k_out=s["k_out"], v_out=s["v_out"])
    return sdpa.sdpa_paged_fwd_fp8(s["q"], *cache, cache_layout=c["order"], max_seqlen_q=s["max_seqlen_q"],
                                   max_seqlen_kv=s["max_seqlen_kv"], mask="causal_br" if c["causal"] else "none",
                                   window=(c["window"], -1), scale=s["scale"], out=s["out"], lse=s["lse"],
                                   workspace=s["workspace"])


# ------------------------------------------------------------------------------------------------ 64 bits
def code_values():
    """The 256 values of E4M3 (bias 7, no infinities), from its bits."""
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v[(b & 127) == 127] = np.nan
    return torch.from_numpy(np.where(b >= 128, -v, v)).to(DEV)


def exact_values(codes, scale):
    return code_values()[codes.int()] * torch.exp2(scale.double() - 127)[..., None]


def exact_quantised(x, c):
    """Rows x (64 bits) as their codes' values and their scales: the least power of two that brings the row under 448, and
    the nearest of the format's values, ties to the even one."""
    lo, hi = LIMITS[c["dtype"]]
    top = x.abs().amax(-1)
    e = torch.ceil(torch.log2(torch.where(top > 0, top, 1.0) / 448.0))
    e = torch.where(top / torch.exp2(e) > 448.0, e + 1, torch.where(top / torch.exp2(e - 1) <= 448.0, e - 1, e))
    scale = torch.exp2(torch.where(top > 0, e.clamp(lo, hi), float(lo)))
    y = (x / scale[..., None]).clamp(-448.0, 448.0)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step, scale


def exact_angles(s):
    """[tokens, rot/2] angles' cosines and sines as complex numbers."""
    half, start, parts = sum(s["sections"]), 0, []
    for n, pos in zip(s["sections"], s["positions"].long()):
        rows = s["cos_sin"][pos].double()
        parts.append(torch.complex(rows[:, start:start + n], rows[:, half + start:half + start + n]))
        start += n
    return torch.cat(parts, dim=1)


def turned(x, turn, pairs):
    """x [rows, heads, d] (64 bits): each pair (a, b) as the complex number a + ib times its token's."""
    rot = 2 * turn.shape[1]
    out = x.clone()
    first = slice(0, rot // 2) if pairs == "half" else slice(0, rot, 2)
    second = slice(rot // 2, rot) if pairs == "half" else slice(1, rot, 2)
    z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn[:, None, :]
    out[..., first], out[..., second] = z.real, z.imag
    return out


def exact_norm(x, weight, turn, pairs):
    x = x.double()
    y = x * torch.rsqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * weight.double()
    return turned(y, turn, pairs)


def exact_norm_back(dy, x, weight, turn, pairs):
    x, d = x.double(), x.shape[-1]
    r = torch.rsqrt((x * x).sum(-1, keepdim=True) / d + EPS)
    g = turned(dy.double(), turn.conj(), pairs)
    h = g * weight.double()
    return r * h - x * r ** 3 * (h * x).sum(-1, keepdim=True) / d, (g * x * r).sum(dim=(0, 1))


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["kind"] == "axes":
        return tuple(exact_norm(s[x], s[x + "_weight"], exact_angles(s), c["pairs"]) for x in ("q", "k"))
    if c["kind"] == "axes_bwd":
        (dq, dwq), (dk, dwk) = (exact_norm_back(s["d%s_out" % x], s[x], s[x + "_weight"], exact_angles(s), c["pairs"])
                                for x in ("q", "k"))
        return dq, dk, dwq, dwk
    cu, lens, tab = s["cu_seqlens_q"].tolist(), s["kv_lens"].tolist(), s["block_table"].cpu().numpy()
    head = torch.arange(c["hkv"], device=DEV)

    def slots(b, lo, hi):  # index of positions [lo, hi) of sequence b, all heads: [hi - lo, hkv]
        pos = np.arange(lo, hi)
        ids, slot = (torch.from_numpy(a.astype(np.int64)).to(DEV)[:, None] for a in (tab[b][pos // c["page"]], pos % c["page"]))
        return (ids, slot, head[None]) if c["order"] == "nhd" else (ids, head[None], slot)

    if c["kind"] == "append8":
        out = [code_values()[s["k_cache"].int()], torch.exp2(s["k_scale"].double() - 127),
               code_values()[s["v_cache"].int()], torch.exp2(s["v_scale"].double() - 127)]
        turn = exact_angles(s) if c["sections"] else None
        q_out = s["q_out"].double() if c["sections"] else None
        for b, n in enumerate(lens):
            lo, hi = cu[b], cu[b + 1]
            if hi == lo:
                continue
            k = s["k"][lo:hi].double()
            if c["sections"]:
                k = exact_norm(k, s["k_weight"], turn[lo:hi], "half")
                q_out[lo:hi] = exact_norm(s["q"][lo:hi], s["q_weight"], turn[lo:hi], "half")
            at = slots(b, n - (hi - lo), n)
            out[0][at], out[1][at] = exact_quantised(k, c)
            out[2][at], out[3][at] = exact_quantised(s["v"][lo:hi].double(), c)
        return out + ([q_out] if c["sections"] else [])
    if c["kind"] == "read8":
        out = [s["k_out"].double(), s["v_out"].double()]
        for b, n in enumerate(lens):
            lo, hi = cu[b], cu[b + 1]
            if hi > lo:
                at = slots(b, n - (hi - lo), n)
                out[0][lo:hi] = exact_values(s["k_cache"][at], s["k_scale"][at])
                out[1][lo:hi] = exact_values(s["v_cache"][at], s["v_scale"][at])
        return out
    o, lse = s["out"].double(), s["lse"].double()
    group = c["hq"] // c["hkv"]
    for b, n in enumerate(lens):
        lo, hi = cu[b], cu[b + 1]
        if hi == lo:
            continue
        at = slots(b, 0, n)
        k, v = exact_values(s["k_cache"][at], s["k_scale"][at]), exact_values(s["v_cache"][at], s["v_scale"][at])
        behind = torch.arange(n - (hi - lo), n, device=DEV)[:, None] - torch.arange(n, device=DEV)[None, :]
        hidden = torch.zeros_like(behind, dtype=torch.bool)
        if c["causal"]:
            hidden = behind < 0
            if c["window"] >= 0:
                hidden |= behind > c["window"]
        for h in range(c["hkv"]):
            x = torch.einsum("qgd,kd->gqk", s["q"][lo:hi, h * group:(h + 1) * group].double(), k[:, h]) * s["scale"]
            x[:, hidden] = -math.inf
            l = torch.logsumexp(x, dim=-1)
            p = torch.exp(x - torch.where(l == -math.inf, 0.0, l)[..., None])
            o[lo:hi, h * group:(h + 1) * group] = torch.einsum("gqk,kd->qgd", p, v[:, h])
            lse[lo:hi, h * group:(h + 1) * group] = l.T
    return o, lse
