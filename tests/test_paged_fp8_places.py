"""Where an 8-bit cache's codes and scale bytes may lie: what the append takes has no
byte in common, counted byte by byte. Only without a GPU: the addresses are made up,
and a call that is not refused ends at the missing device."""
import itertools
import random

import numpy as np
import pytest
import torch

from test_paged_abi import BASE, M, built, paged_problem  # noqa: F401 (built: the module's fixture)
from test_paged_fp8_abi import append, scales

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="takes calls with made-up addresses")
OVERLAP = 4
TENSORS = ("k", "v", "k_scale", "v_scale")


def call(pages, heads, at, strides):
    """The append's answer; at, strides: of each tensor, its first byte behind BASE + 8 M and (page, slot, head)."""
    names = ("page", "slot", "head")
    codes = {f"{t}_{n}_stride": s for t in "kv" for n, s in zip(names, strides[t])}
    bytes_ = {f"{t}_{n}_stride": s for t in "kv" for n, s in zip(names, strides[t + "_scale"])}
    p = paged_problem(num_pages=pages, num_heads_kv=heads, num_heads_q=heads, total_q=1, seqlen_q=1, **codes)
    base = BASE + 8 * M
    return append(p, s=scales(k=base + at["k_scale"], v=base + at["v_scale"], **bytes_), kc=base + at["k"], vc=base + at["v"])


def bytes_of(pages, heads, at, strides, width):
    g, s, h, x = np.meshgrid(np.arange(pages), np.arange(16), np.arange(heads), np.arange(width), indexing="ij")
    return (at + g * strides[0] + s * strides[1] + h * strides[2] + x).ravel()


def share_bytes(pages, heads, at, strides):
    every = [bytes_of(pages, heads, at[t], strides[t], 1 if "scale" in t else 128) for t in TENSORS]
    every = np.concatenate(every)
    return len(np.unique(every)) < len(every)


def far(**kw):
    """Four tensors apart, with some places replaced."""
    at = dict(k=0, v=M, k_scale=2 * M, v_scale=3 * M)
    strides = dict(k=(8192, 512, 128), v=(8192, 512, 128), k_scale=(32, 2, 1), v_scale=(32, 2, 1))
    for name, (a, s) in kw.items():
        at[name], strides[name] = a, s or strides[name]
    return at, strides


def test_steps_that_do_not_divide_a_larger_stride():
    """Places that lie apart modulo the slots' step, but not modulo the pages'."""
    assert call(2, 2, *far()) != OVERLAP
    for kw in (dict(k_scale=(256, (8448, 512, 1))),                  # scales in K's gaps, pages 33 slots long
               dict(v_scale=(256, (8448, 512, 1))),
               dict(v_scale=(M + 256, (8448, 512, 1))),              # in V's
               dict(k_scale=(2 * M, (64, 4, 1)), v_scale=(2 * M + 2, (66, 4, 1)))):  # each other's
        at, strides = far(**kw)
        assert share_bytes(2, 2, at, strides)
        assert call(2, 2, at, strides) == OVERLAP, kw
    # the same places with pages of whole slots, and of whole pages
    for page in (8192, 16384):
        at, strides = far(k_scale=(256, (page, 512, 1)))
        shared = share_bytes(2, 2, at, strides)
        assert not shared and call(2, 2, at, strides) != OVERLAP


@pytest.mark.parametrize("heads", [1, 2, 3])
def test_blocks_are_taken(heads):
    """Codes and scale bytes of a page, of a slot, or of a head in one block."""
    n = 16 * heads
    page = 2 * n * 128 + heads * 128 * 16
    at, strides = far(k=(0, (page, heads * 128, 128)), v=(n * 128, (page, heads * 128, 128)),
                      k_scale=(2 * n * 128, (page, heads, 1)), v_scale=(2 * n * 128 + n, (page, heads, 1)))
    assert not share_bytes(3, heads, at, strides) and call(3, heads, at, strides) != OVERLAP
    slot = 2 * heads * 128 + heads * 128
    at, strides = far(k=(0, (16 * slot, slot, 128)), v=(heads * 128, (16 * slot, slot, 128)),
                      k_scale=(2 * heads * 128, (16 * slot, slot, 1)), v_scale=(2 * heads * 128 + heads, (16 * slot, slot, 1)))
    assert not share_bytes(3, heads, at, strides) and call(3, heads, at, strides) != OVERLAP
    head = 2 * 128 + 16
    at, strides = far(k=(0, (16 * heads * head, heads * head, head)), v=(128, (16 * heads * head, heads * head, head)),
                      k_scale=(256, (16 * heads * head, heads * head, head)),
                      v_scale=(257, (16 * heads * head, heads * head, head)))
    assert not share_bytes(3, heads, at, strides) and call(3, heads, at, strides) != OVERLAP


def test_whatever_is_taken_shares_no_byte():
    rng = random.Random(5)
    taken = shared = 0
    for _ in range(400):
        pages, heads = rng.choice([1, 2, 3]), rng.choice([1, 2, 3])
        pad = rng.choice([0, 16, 128])
        head = 128 + pad
        slot = heads * head * rng.choice([1, 1, 2, 3])
        page = 16 * slot * rng.choice([1, 1, 2])
        codes = (page, slot, head)
        if heads > 1 and rng.random() < 0.3:  # [page][head][slot]
            codes = (page, head, 16 * head * (slot // (heads * head)))
        at = dict(k=0, v=rng.choice([head, heads * head, slot * 16, 128, page * 4, rng.randrange(0, 3 * page, 16)]))
        strides = dict(k=codes, v=codes)
        for t in ("k_scale", "v_scale"):
            s = [rng.choice([codes[i], codes[i], codes[i] + rng.choice([1, 16, 128, 256]), d]) for i, d in
                 enumerate((16 * heads, heads, 1))]
            strides[t] = tuple(s)
            at[t] = rng.choice([128, head * heads - 1, rng.randrange(0, 2 * page), rng.randrange(0, page * (pages + 1)), 9 * page])
        got = call(pages, heads, at, strides)
        if share_bytes(pages, heads, at, strides):
            shared += 1
            assert got == OVERLAP, (pages, heads, at, strides)
        taken += got != OVERLAP
    assert taken > 15 and shared > 100  # both kinds are met


def test_pairs():
    """Every pair of tensors in one place is refused."""
    for a, b in itertools.combinations(TENSORS, 2):
        at, strides = far()
        at[b] = at[a]
        assert call(2, 2, at, strides) == OVERLAP, (a, b)
