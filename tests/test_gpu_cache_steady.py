"""The operators around the 8-bit cache where a warp or block does the same thing many times over:
places of rings used again, tables of angles written anew, heads one after another, pieces
after pieces. Against the 64-bit references, with the tolerances of test_gpu_cache."""
import math

import pytest
import torch

import prefill_kda_chunk_gb300 as K
from oracle import cache as C
from test_gpu_cache import (BF16, F32, F8, I32, attention_close, built, cache_case, close, cu_of, deal,  # noqa: F401
                            empty_cache, heads_case, i32, make, same_cache)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------- norms and rotation

# A GPU takes 2432 warps at a time. Tokens (or parts of a token's heads) that a warp of the forward
# kernel comes to, and batches of its ring of three in brackets; batches of one of the gradient.
STEADY = [
    (6000, 3, 1, 64, 64, False, True, 1 << 20),      # 3 (6); 5
    (6000, 3, 1, 64, 32, True, True, 70000),         # the same, by pairs
    (3001, 16, 3, 128, 128, False, True, 5000),      # 3 halves (6); 6
    (3001, 16, 3, 128, 64, True, False, 1 << 22),
    (5000, 5, 2, 256, 256, False, True, 100),        # 3 (9); 8
    (5000, 5, 2, 256, 96, True, True, 1 << 24),
    (2600, 64, 8, 128, 128, False, True, 100000),    # 5 quarters (15); 19
    (20000, 1, 0, 64, 48, False, False, 300),        # 9 (9); 8
    (9000, 7, 1, 128, 0, False, True, 0),            # 4 (8); 11, nothing turned
    (8192, 64, 8, 128, 128, False, True, 0),         # 7 halves (35); 61
]


@pytest.mark.parametrize("T,Hq,Hk,D,R,pairs,fused,far", STEADY)
def test_norms_of_many_tokens(T, Hq, Hk, D, R, pairs, fused, far):
    _, q, k, w, freq, pos = heads_case(T, Hq, Hk, D, R, pairs, fused, far, seed=1)
    qo, ko = K.qk_norm_rope(q, k, *w, freq, pos, interleaved=pairs)
    K.check_device_error()
    close(qo, *C.norm_rope(q, w[0], freq, pos, interleaved=pairs), "q")
    if Hk:
        close(ko, *C.norm_rope(k, w[1], freq, pos, interleaved=pairs), "k")
    K.qk_norm_rope(q, k, *w, freq, pos, interleaved=pairs, q_out=q, k_out=k)
    assert torch.equal(q, qo) and (k is None or torch.equal(k, ko)), "in place"


@pytest.mark.parametrize("d32", [True, False])
@pytest.mark.parametrize("T,Hq,Hk,D,R,pairs,fused,far", STEADY)
def test_gradients_of_many_tokens(T, Hq, Hk, D, R, pairs, fused, far, d32):
    r, q, k, w, freq, pos = heads_case(T, Hq, Hk, D, R, pairs, fused, far, seed=2)
    dtype = F32 if d32 else BF16
    dy = r(T, (Hq + Hk) * D, dtype=dtype)
    dqo = dy[:, :Hq * D].unflatten(1, (Hq, D))
    dko = dy[:, Hq * D:].unflatten(1, (Hk, D)) if Hk else None
    got = K.qk_norm_rope_backward(q, k, dqo, dko, *w, freq, pos, interleaved=pairs)
    K.check_device_error()
    for x, dyo, wi, d, dw, name in ((q, dqo, w[0], got[0], got[2], "q"), (k, dko, w[1], got[1], got[3], "k")):
        if x is None:
            continue
        rx, rw = C.norm_rope_backward(x, dyo, wi, freq, pos, interleaved=pairs)
        close(d, *rx, "d" + name)
        close(dw, *rw, f"d{name}_weight")


# ----------------------------------------------------------- into the cache

# D, page, key-value heads: warps of an item (kept rows a lane), heads of an item and its sets of them.
HEADS_TOGETHER = [
    (128, 8, 9),      # 1 (4), 8 + 1
    (64, 16, 5),      # 1 (4), 4 + 1
    (128, 8, 3),      # 1 (4), 2 + 1
    (128, 16, 5),     # 2 (4), 4 + 1
    (64, 32, 9),      # 2 (4), 8 + 1
    (128, 32, 9),     # 4 (4), 8 + 1
    (64, 64, 3),      # 4 (4), 2 + 1
    (128, 64, 9),     # 8 (4), 8 + 1
    (128, 50, 6),     # 8 (4), 4 + 2
    (64, 128, 5),     # 8 (4), 4 + 1
    (128, 128, 9),    # 8 (8), 8 + 1
    (128, 200, 4),    # 8 (8), 2 + 2; rows behind those in registers
]


@pytest.mark.parametrize("D,page,H,layout", [(*c, ("page", "heads first")[i % 2]) for i, c in enumerate(HEADS_TOGETHER)])
def test_append_of_several_heads_an_item(D, page, H, layout):
    """Prompts, then more tokens for the same slots: pages that go on, whose scales grow in some of an
    item's heads and not in the next; infinities and NaN in some heads only, the first and
    the last among them."""
    g = torch.Generator().manual_seed(D + page + H)
    # (24 warps for every SM with all sets of heads: what the items' number goes by)
    w = next(w for w in (1, 2, 4, 8) if page <= 4 * (256 // D) * w or w == 8)
    B, want = 40, -(-24 * 152 // (2 * 2 * w)) * page
    rounds = [torch.randint(1, 3 * page, (B,), generator=g).tolist(),
              [want // B + int(x) for x in torch.randint(0, page, (B,), generator=g)]]
    ends = [sum(r[i] for r in rounds) for i in range(B)]
    table, pages = deal(ends, page, 2, B + page)
    dev = empty_cache(pages, page, H, D, layout)
    ref = [(c.cpu().double(), s.cpu().double()) for c, s in ((dev[0], dev[2]), (dev[1], dev[3]))]
    r, lens = make(D + page + H), [0] * B
    for n, new in enumerate(rounds):
        lens = [a + b for a, b in zip(lens, new)]
        T = sum(new)
        x = r(T, 2, H, D)
        x *= torch.exp2(torch.randint(-3, 3, (T, 1, 1, 1), device="cuda").float())
        # the heads' sizes go up, stay, or go down from one round to the next
        x *= torch.exp2((n * (torch.arange(H, device="cuda") % 3 - 1) * 5.0))[None, None, :, None]
        for i in range(24):
            at, h = int(torch.randint(0, T, (1,), generator=g)), (0, H - 1, int(torch.randint(0, H, (1,), generator=g)))[i % 3]
            x[at, i % 2, h, i] = (math.inf, -math.inf, math.nan)[i % 3 - (i > 11)]
        cu = cu_of(new)
        K.paged_append_fp8(x[:, 0], x[:, 1], *dev, table.cuda(), i32(lens), cu.cuda())
        K.check_device_error()
        for y, (codes, scale) in zip((x[:, 0], x[:, 1]), ref):
            C.append(y, codes, scale, table, lens, cu)
        same_cache(dev, ref)


def test_append_of_several_heads_a_token_each():
    """Enough slots that a token each is taken by items of several heads."""
    B, H, D, page = 700, 11, 64, 4
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 9, (B,), generator=g).tolist()
    table, pages = deal([n + 1 for n in lens], page, 1, 1)
    dev = empty_cache(pages, page, H, D, "page")
    for c, s in ((dev[0], dev[2]), (dev[1], dev[3])):
        c.view(torch.uint8).copy_(torch.randint(0, 120, c.shape, generator=g, dtype=torch.uint8))
        s.copy_(torch.exp2(torch.randint(-9, -4, s.shape, generator=g).float()))
    ref = [(c.cpu().double(), s.cpu().double()) for c, s in ((dev[0], dev[2]), (dev[1], dev[3]))]
    new = [n + 1 if i % 7 else 0 for i, n in enumerate(lens)]   # (some without)
    x = make(8)(B, 2, H, D)
    K.paged_append_fp8(x[:, 0], x[:, 1], *dev, table.cuda(), i32(new))
    K.check_device_error()
    for y, (codes, scale) in zip((x[:, 0], x[:, 1]), ref):
        C.append(y, codes, scale, table, new)
    same_cache(dev, ref)


# -------------------------------------------------------------- the attention

# Tiles of 128 tokens that each of 152 blocks takes (more than twice the places for keys, of which there
# are 5, 6 or, with 64 channels, 10): 16 to 17, or 27 to 28.
@pytest.mark.parametrize("lens,Hq,Hkv,D,page,layout", [
    ([69000, 9000, 0, 2500], 64, 4, 128, 64, "page"),            # 16 heads
    ([69000, 9000, 0, 2500], 64, 4, 128, 17, "heads first"),     # copies by threads
    ([70000, 11, 8500], 32, 4, 128, 17, "token"),                # 8 heads
    ([110000, 21000, 3], 64, 4, 64, 32, "heads first"),
    ([110000, 21000, 3], 64, 4, 64, 17, "page"),
    ([7, 130000, 2500], 20, 4, 64, 8, "page"),
    ([130000, 2500], 32, 4, 64, 17, "apart"),
])
def test_decode_of_many_tiles_a_block(lens, Hq, Hkv, D, page, layout):
    case = cache_case(lens, Hq, Hkv, D, page, layout, seed=11, spread=1)
    o, l = K.paged_decode_fp8(*case)
    K.check_device_error()
    attention_close(o, l, *case[:6], lens)


# A block's pieces, whole items and parts of them: 10 to 11, of 3 or 4 places for queries.
@pytest.mark.parametrize("Hq,Hkv,D,page", [(32, 8, 128, 16), (128, 8, 128, 64), (64, 8, 64, 17), (96, 8, 64, 32),
                                           (128, 8, 128, 17)])
def test_decode_of_many_pieces_a_block(Hq, Hkv, D, page):
    g = torch.Generator().manual_seed(Hq + D + page)
    lens = torch.randint(1, 301, (200,), generator=g).tolist()
    lens[3] = lens[199] = 0
    case = cache_case(lens, Hq, Hkv, D, page, seed=12, spread=1)
    o, l = K.paged_decode_fp8(*case)
    K.check_device_error()
    attention_close(o, l, *case[:6], lens)
