"""Measured cases of the serving and training operators around the attention kernels: the per-head norm and
rotation of queries and keys with its gradient, the write of new keys and values into a paged cache, and the
attention of new tokens over that cache.

`run` computes them in their plain form (elementary torch operations, 32 bits, rounded once), or, where `own` is
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
EPS = 1e-6
THETA = 10000.0
WORKSPACE_BYTES = 256 << 20  # scratch that a serving program keeps for its attention calls


# ------------------------------------------------------------------------------------------------ cases
def norm_case(name, kind, tokens, hq, hkv, d, rot, pairs, dtype, fused, max_pos):
    """rot: leading values of a head that are rotated; pairs: "half" (i, i + rot/2) or "adjacent" (2i, 2i+1);
    fused: q and k are slices of one projection's output rows."""
    return dict(name=name, kind=kind, tokens=tokens, hq=hq, hkv=hkv, d=d, rot=rot, pairs=pairs, dtype=dtype, fused=fused,
                max_pos=max_pos)


def cache_case(name, kind, batch, q_lo, q_hi, kv_lo, kv_hi, hq, hkv, d, dv, page, order, dtype, window=-1, causal=True, pad=0,
               rot=0):
    """A batch whose new tokens number q_lo..q_hi and whose total lengths, those tokens among them, kv_lo..kv_hi, evenly
    spaced; order: "nhd" pages hold [slot][head][d], "hnd" [head][slot][d]; window: keys left of the diagonal, -1 all;
    pad: rows behind the last sequence; append: rot > 0 norms q and k and rotates their leading values on the way."""
    return dict(name=name, kind=kind, batch=batch, q_lo=q_lo, q_hi=q_hi, kv_lo=kv_lo, kv_hi=kv_hi, hq=hq, hkv=hkv, d=d, dv=dv,
                page=page, order=order, dtype=dtype, window=window, causal=causal, pad=pad, rot=rot)


def listed():
    return [
        # one decode step of a few sequences: latency
        norm_case("norm_rope_step", "norm", 4, 32, 8, 128, 128, "half", "bf16", True, 8192),
        # a prefill or training step's tokens, straight from the fused projection
        norm_case("norm_rope_train", "norm", 18000, 32, 8, 128, 128, "half", "bf16", True, 8192),
        # half of a 256-wide head rotated, adjacent pairs, odd token count
        norm_case("norm_rope_bwd_d256", "norm_bwd", 4099, 16, 8, 256, 128, "adjacent", "fp16", False, 8192),
        # the gradient for a training step's tokens
        norm_case("norm_rope_bwd_train", "norm_bwd", 18000, 32, 8, 128, 128, "half", "bf16", True, 8192),
        # decode: every sequence appends one token, normed and rotated on the way
        cache_case("append_step", "append", 33, 1, 1, 1, 1000, 32, 8, 128, 128, 16, "nhd", "bf16", rot=128),
        # prefill chunks of uneven length copied into pages of another head order
        cache_case("append_chunk_d256", "append", 7, 1, 4001, 9, 6007, 16, 8, 256, 256, 64, "hnd", "bf16"),
        # one user's next token over a short context: latency
        cache_case("decode_one", "paged", 1, 1, 1, 999, 999, 32, 8, 128, 128, 16, "nhd", "bf16"),
        # a serving batch of uneven contexts, one token each
        cache_case("decode_batch", "paged", 64, 1, 1, 500, 16384, 32, 8, 128, 128, 16, "nhd", "bf16", pad=3),
        # sliding-window layer of the same kind of batch
        cache_case("decode_window_d256", "paged", 48, 1, 1, 1, 8192, 16, 8, 256, 256, 64, "hnd", "fp16", window=1024),
        # one long prompt's next chunk over what is cached already
        cache_case("chunk_long", "paged", 1, 2048, 2048, 16384, 16384, 32, 8, 128, 128, 32, "nhd", "bf16"),
        # prompts' chunks and decoding sequences in one batch, 512-wide heads of a global layer
        cache_case("mixed_d512", "paged", 6, 1, 509, 700, 6000, 16, 4, 512, 512, 128, "nhd", "bf16"),
        # wide query/key heads with narrower value heads, a few speculative tokens each, all keys seen
        cache_case("spec_d192", "paged", 9, 0, 5, 5, 4097, 32, 8, 192, 128, 48, "nhd", "bf16", causal=False),
    ]


def spread(rng, lo, hi):
    """A whole number of [lo, hi], its logarithm uniform."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        k = "norm" if c["kind"].startswith("norm") else c["kind"]
        most[k] = {x: max(most.get(k, {}).get(x, 0), w[x]) for x in ("bytes", "flops")}
    while True:
        kind = rng.choice(["norm", "norm_bwd", "append", "paged", "paged", "paged"])
        d = rng.choice([128, 128, 128, 256, 512, 192])
        hq, hkv = rng.choice([(32, 8), (16, 8), (16, 4), (16, 16), (8, 1), (14, 2), (10, 10), (32, 1)])
        dtype = rng.choice(["bf16", "fp16"])
        if kind in ("norm", "norm_bwd"):
            c = norm_case("", kind, spread(rng, 1, 18000), hq, hkv, d, rng.choice([d, d, d // 2, 64, 0]),
                          rng.choice(["half", "adjacent"]), dtype, rng.random() < 0.5, 8192)
        else:
            q_hi = rng.choice([1, 1, spread(rng, 2, 16), spread(rng, 16, 2048)])
            kv_hi = spread(rng, max(q_hi, 8), 16384)
            c = cache_case("", kind, spread(rng, 1, 100), rng.choice([min(1, q_hi), 0, q_hi]), q_hi,
                           max(1, int(kv_hi * rng.random())), kv_hi, hq, hkv, d, 128 if d == 192 else d,
                           rng.choice([16, 32, 64, 128, 256, 48]), rng.choice(["nhd", "hnd"]), dtype,
                           rng.choice([-1, -1, spread(rng, 1, 4096)]) if kind == "paged" else -1,
                           kind == "append" or rng.random() < 0.8, rng.choice([0, 0, spread(rng, 1, 100)]),
                           rng.choice([0, d, 64]) if kind == "append" else 0)
            if not c["causal"]:
                c["window"] = -1
            elems = c["batch"] * kv_hi * max(hkv * d, hq * q_hi)  # the plain form pads every sequence to the longest
            if elems > 1.2e9 or sum(q for q, _ in lengths(c)) == 0:
                continue
        w = work(c)
        if all(w[x] <= most["norm" if kind.startswith("norm") else kind][x] for x in w):
            del c["name"]
            return c


def lengths(c):
    """(new tokens, total length) of every sequence, before the seed shuffles their order."""
    n = c["batch"]
    at = [i / (n - 1) if n > 1 else 1.0 for i in range(n)]
    total = [c["kv_lo"] + round((c["kv_hi"] - c["kv_lo"]) * f) for f in at]
    order = sorted(range(n), key=lambda i: (i * 7919) % n if math.gcd(7919, n) == 1 else i)
    new = [c["q_lo"] + round((c["q_hi"] - c["q_lo"]) * at[i]) for i in order]
    return [(q, max(q, k)) for q, k in zip(new, total)]


def work(c):
    if c["kind"] in ("norm", "norm_bwd"):
        rows, heads = c["tokens"], c["hq"] + c["hkv"]
        moved = 2 if c["kind"] == "norm" else 3
        extra = rows * (4 * c["rot"] + 4) + (2 if c["kind"] == "norm" else 2 + 4) * 2 * c["d"]
        return {"bytes": moved * 2 * rows * heads * c["d"] + extra,
                "flops": (8 if c["kind"] == "norm" else 18) * rows * heads * c["d"]}
    seqs = lengths(c)
    new = sum(q for q, _ in seqs)
    if c["kind"] == "append":
        moved = c["hkv"] * (c["d"] + c["dv"]) + (c["hq"] * c["d"] if c["rot"] else 0)
        return {"bytes": 4 * new * moved + new * (4 + 4 * c["rot"]) + 8 * c["batch"],
                "flops": 8 * new * (c["hq"] + c["hkv"]) * c["d"] if c["rot"] else 0}
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
    return {"bytes": 2 * kv_rows * c["hkv"] * (c["d"] + c["dv"]) + new * c["hq"] * (2 * c["d"] + 2 * c["dv"] + 4)
            + 4 * sum(-(-k // c["page"]) for q, k in seqs if q) + 8 * c["batch"],
            "flops": 2 * pairs * c["hq"] * (c["d"] + c["dv"])}


# ------------------------------------------------------------------------------------------------ inputs
def table(max_pos, rot):
    """[max_pos, rot] float32: rot/2 cosines, then rot/2 sines of position * THETA^(-2i/rot)."""
    if rot == 0:
        return torch.zeros((max_pos, 0), device=DEV)
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


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV).manual_seed(seed * 2 + 1)
    rng = np.random.default_rng(seed)
    dt, d = DTYPES[c["dtype"]], c["d"]
    s = {"case": c}
    if c["kind"] in ("norm", "norm_bwd") or c["rot"]:
        s["q_weight"], s["k_weight"] = normal(gen, (d,), dt, 1.0, 0.2), normal(gen, (d,), dt, 1.0, 0.2)
    if c["kind"] in ("norm", "norm_bwd"):
        s["q"], s["k"] = projected(gen, c["tokens"], c, [(c["hq"], d), (c["hkv"], d)])
        s["cos_sin"] = table(c["max_pos"], c["rot"])
        s["positions"] = torch.from_numpy(rng.integers(0, c["max_pos"], c["tokens"]).astype(np.int32)).to(DEV)
        if c["kind"] == "norm_bwd":
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
    shape = lambda w: (pages, c["page"], c["hkv"], w) if c["order"] == "nhd" else (pages, c["hkv"], c["page"], w)  # noqa: E731
    s["k_cache"], s["v_cache"] = normal(gen, shape(d), dt), normal(gen, shape(c["dv"]), dt)
    if c["kind"] == "append":
        s["q"], s["k"], s["v"] = projected(gen, rows, c, [(c["hq"], d), (c["hkv"], d), (c["hkv"], c["dv"])])
        if c["rot"]:
            s["cos_sin"] = table(s["max_seqlen_kv"], c["rot"])
            s["q_out"] = torch.zeros((rows, c["hq"], d), dtype=dt, device=DEV)
    else:
        s["q"] = normal(gen, (rows, c["hq"], d), dt)
        s["out"] = torch.zeros((rows, c["hq"], c["dv"]), dtype=dt, device=DEV)
        s["lse"] = torch.zeros((rows, c["hq"]), device=DEV)
        s["workspace"] = torch.empty(WORKSPACE_BYTES, dtype=torch.uint8, device=DEV)
        s["scale"] = d ** -0.5
    return s


# ------------------------------------------------------------------------------------------------ plain forms
def rotate(x, cos_sin, pairs, back=False):
    """x [rows, heads, d] with its leading values rotated by their row's angles (backwards: by the negative)."""
    rot = cos_sin.shape[1]
    if rot == 0:
        return x
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
    """Sequence, position and liveness of every query row."""
    cu, at = s["cu_seqlens_q"].long(), torch.arange(rows, device=DEV)
    seq = torch.clamp((at[:, None] >= cu[None, 1:]).sum(1), max=cu.numel() - 2)
    new = cu[seq + 1] - cu[seq]
    return seq, s["kv_lens"].long()[seq] - new + (at - cu[seq]), at < cu[-1]


def run_paged(s, c):
    cu, lens = s["cu_seqlens_q"].long(), s["kv_lens"].long()
    hq, hkv, page = c["hq"], c["hkv"], c["page"]
    key = torch.arange(s["max_seqlen_kv"], device=DEV)
    ids = s["block_table"].long().clamp(min=0)[:, key // page]
    there = key[None, :] < lens[:, None]                                              # [batch, keys]

    def gather(cache):                                                                # [batch, hkv, keys, width]
        rows = cache[ids, key % page] if c["order"] == "nhd" else cache.transpose(1, 2)[ids, key % page]
        return (rows.float() * there[:, :, None, None]).transpose(1, 2)

    i = torch.arange(s["max_seqlen_q"], device=DEV)
    new = cu[1:] - cu[:-1]
    row = (cu[:-1, None] + i[None, :]).clamp(max=max(s["q"].shape[0] - 1, 0))
    live = i[None, :] < new[:, None]                                                  # [batch, queries]
    q = s["q"][row].float().unflatten(2, (hkv, hq // hkv)).permute(0, 2, 3, 1, 4)      # [batch, hkv, group, queries, d]
    score = torch.matmul(q.flatten(2, 3), gather(s["k_cache"]).transpose(2, 3)).unflatten(2, (hq // hkv, -1)) * s["scale"]
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
    o = torch.matmul(p.flatten(2, 3), gather(s["v_cache"])).unflatten(2, (hq // hkv, -1))
    o = o / torch.where(total == 0, torch.ones_like(total), total)
    lse = (top + torch.log(total)).squeeze(-1)
    s["out"][row[live]] = o.permute(0, 3, 1, 2, 4).flatten(2, 3)[live].to(s["out"].dtype)
    s["lse"][row[live]] = lse.permute(0, 3, 1, 2).flatten(2, 3)[live]
    return s["out"], s["lse"]


def run_append(s, c):
    rows = s["k"].shape[0]
    seq, pos, live = places(s, rows)
    k, v = s["k"], s["v"]
    if c["rot"]:
        angles = s["cos_sin"][pos.clamp(0, s["cos_sin"].shape[0] - 1)]
        k = norm(k, s["k_weight"], angles, "half").to(k.dtype)
        s["q_out"][live] = norm(s["q"], s["q_weight"], angles, "half").to(k.dtype)[live]
    seq, pos = seq[live], pos[live]
    ids, slot = s["block_table"].long()[seq, pos // c["page"]], pos % c["page"]
    for cache, x in ((s["k_cache"], k), (s["v_cache"], v)):
        (cache if c["order"] == "nhd" else cache.transpose(1, 2))[ids, slot] = x[live]
    return [s["k_cache"], s["v_cache"]] + ([s["q_out"]] if c["rot"] else [])


def run(state):
    s, c = state, state["case"]
    if own:
        return run_own(s, c)
    if c["kind"] == "norm":
        angles, dt = s["cos_sin"][s["positions"].long()], s["q"].dtype
        return (norm(s["q"], s["q_weight"], angles, c["pairs"]).to(dt), norm(s["k"], s["k_weight"], angles, c["pairs"]).to(dt))
    if c["kind"] == "norm_bwd":
        angles, dt = s["cos_sin"][s["positions"].long()], s["q"].dtype
        dq, dwq = norm_back(s["dq_out"], s["q"], s["q_weight"], angles, c["pairs"])
        dk, dwk = norm_back(s["dk_out"], s["k"], s["k_weight"], angles, c["pairs"])
        return dq.to(dt), dk.to(dt), dwq, dwk
    return run_append(s, c) if c["kind"] == "append" else run_paged(s, c)


def run_own(s, c):
    import scaled_dot_product_02_gb300 as sdpa

    if c["kind"] == "norm":
        return sdpa.sdpa_qk_norm_rope(s["q"], s["k"], s["q_weight"], s["k_weight"], s["cos_sin"], s["positions"], eps=EPS,
                                      interleaved=c["pairs"] == "adjacent")
    if c["kind"] == "norm_bwd":
        return sdpa.sdpa_qk_norm_rope_bwd(s["dq_out"], s["dk_out"], s["q"], s["k"], s["q_weight"], s["k_weight"], s["cos_sin"],
                                          s["positions"], eps=EPS, interleaved=c["pairs"] == "adjacent")
    if c["kind"] == "append":
        if not c["rot"]:
            sdpa.sdpa_paged_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["block_table"], s["kv_lens"],
                                   s["cu_seqlens_q"], cache_layout=c["order"])
            return [s["k_cache"], s["v_cache"]]
        sdpa.sdpa_paged_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["block_table"], s["kv_lens"], s["cu_seqlens_q"],
                               cache_layout=c["order"], q=s["q"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                               cos_sin=s["cos_sin"], eps=EPS, q_out=s["q_out"])
        return [s["k_cache"], s["v_cache"], s["q_out"]]
    return sdpa.sdpa_paged_fwd(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["kv_lens"], s["cu_seqlens_q"],
                               cache_layout=c["order"], max_seqlen_q=s["max_seqlen_q"], max_seqlen_kv=s["max_seqlen_kv"],
                               mask="causal_br" if c["causal"] else "none", window=(c["window"], -1), scale=s["scale"],
                               out=s["out"], lse=s["lse"], workspace=s["workspace"])


# ------------------------------------------------------------------------------------------------ 64 bits
def turned(x, angles, pairs, sign):
    """x [rows, heads, d] (64 bits): each pair (a, b) as the complex number a + ib times cos + i sign sin."""
    rot = angles.shape[1]
    turn = torch.complex(angles[:, :rot // 2].double(), sign * angles[:, rot // 2:].double())[:, None, :]
    out = x.clone()
    first = slice(0, rot // 2) if pairs == "half" else slice(0, rot, 2)
    second = slice(rot // 2, rot) if pairs == "half" else slice(1, rot, 2)
    z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn
    out[..., first], out[..., second] = z.real, z.imag
    return out


def exact_norm(x, weight, angles, pairs):
    x = x.double()
    y = x * torch.rsqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * weight.double()
    return turned(y, angles, pairs, 1.0)


def exact_norm_back(dy, x, weight, angles, pairs):
    x, d = x.double(), x.shape[-1]
    r = torch.rsqrt((x * x).sum(-1, keepdim=True) / d + EPS)
    g = turned(dy.double(), angles, pairs, -1.0)
    h = g * weight.double()
    return r * h - x * r ** 3 * (h * x).sum(-1, keepdim=True) / d, (g * x * r).sum(dim=(0, 1))


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["kind"] == "norm":
        angles = s["cos_sin"][s["positions"].long()]
        return tuple(exact_norm(s[x], s[x + "_weight"], angles, c["pairs"]) for x in ("q", "k"))
    if c["kind"] == "norm_bwd":
        angles = s["cos_sin"][s["positions"].long()]
        (dq, dwq), (dk, dwk) = (exact_norm_back(s["d%s_out" % x], s[x], s[x + "_weight"], angles, c["pairs"]) for x in ("q", "k"))
        return dq, dk, dwq, dwk
    cu, lens, tab = s["cu_seqlens_q"].tolist(), s["kv_lens"].tolist(), s["block_table"].cpu().numpy()
    if c["kind"] == "append":
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        q_out = s["q_out"].double() if c["rot"] else None
        for b, n in enumerate(lens):
            lo, hi = cu[b], cu[b + 1]
            if hi == lo:
                continue
            pos = np.arange(n - (hi - lo), n)
            ids, slot = (torch.from_numpy(a.astype(np.int64)).to(DEV) for a in (tab[b][pos // c["page"]], pos % c["page"]))
            k = s["k"][lo:hi].double()
            if c["rot"]:
                angles = s["cos_sin"][torch.from_numpy(pos).to(DEV)]
                k = exact_norm(k, s["k_weight"], angles, "half")
                q_out[lo:hi] = exact_norm(s["q"][lo:hi], s["q_weight"], angles, "half")
            head = torch.arange(c["hkv"], device=DEV)
            at = (ids[:, None], slot[:, None], head[None]) if c["order"] == "nhd" else (ids[:, None], head[None], slot[:, None])
            kc[at], vc[at] = k, s["v"][lo:hi].double()
        return [kc, vc] + ([q_out] if c["rot"] else [])
    o, lse = s["out"].double(), s["lse"].double()
    group = c["hq"] // c["hkv"]
    for b, n in enumerate(lens):
        lo, hi = cu[b], cu[b + 1]
        if hi == lo:
            continue
        ids = torch.from_numpy(tab[b, :-(-n // c["page"])].astype(np.int64)).to(DEV)
        k, v = s["k_cache"][ids], s["v_cache"][ids]
        if c["order"] == "hnd":
            k, v = k.transpose(1, 2), v.transpose(1, 2)
        k, v = k.flatten(0, 1)[:n], v.flatten(0, 1)[:n]
        behind = torch.arange(n - (hi - lo), n, device=DEV)[:, None] - torch.arange(n, device=DEV)[None, :]
        hidden = torch.zeros_like(behind, dtype=torch.bool)
        if c["causal"]:
            hidden = behind < 0
            if c["window"] >= 0:
                hidden |= behind > c["window"]
        for h in range(c["hkv"]):
            x = torch.einsum("qgd,kd->gqk", s["q"][lo:hi, h * group:(h + 1) * group].double(), k[:, h].double()) * s["scale"]
            x[:, hidden] = -math.inf
            l = torch.logsumexp(x, dim=-1)
            p = torch.exp(x - torch.where(l == -math.inf, 0.0, l)[..., None])
            o[lo:hi, h * group:(h + 1) * group] = torch.einsum("gqk,kd->qgd", p, v[:, h].double())
            lse[lo:hi, h * group:(h + 1) * group] = l.T
    return o, lse
