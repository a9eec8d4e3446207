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
