"""Page plans, norms of queries and keys with the rotation, the 8-bit cache and the
attention over it, on the GPU, against the 64-bit references.

Tolerances, element by element. A bf16 output is rounded once, by at most 2^-8 of its
value; before that it is a sum whose terms have an absolute sum S, known from the
reference, and whose arithmetic errs by far less than 2^-12 S: fp32 operations of 2^-24
each, angles to 2^-20 of a turn, and in the attention weights of 16 bits. An fp32 sum is
allowed 2^-17 S. Whole numbers, and what the cache holds, are exact.
"""
import math
import threading

import pytest
import torch

import prefill_kda_chunk_gb300 as K
from oracle import cache as C

pytestmark = pytest.mark.gpu

BF16, F32, F8, I32 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.int32


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from prefill_kda_chunk_gb300 import build
    build.build()
    K.lib()


def close(got, ref, size, tag):
    got = got.detach().cpu()
    coarse = got.dtype == BF16
    got = got.double()
    assert torch.isfinite(got).all(), f"{tag}: not finite"
    tol = (2.0 ** -8 * ref.abs() + 2.0 ** -12 * size) if coarse else 2.0 ** -17 * size
    worst = ((got - ref).abs() - tol).max() if got.numel() else torch.tensor(-1.0)
    assert worst <= 1e-30, f"{tag}: over the bound by {float(worst):.3e}"


def make(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, dtype=BF16, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)
    return randn


def i32(v):
    return torch.tensor(v, dtype=I32, device="cuda")


def cu_of(lens):
    return torch.tensor([0] + list(lens)).cumsum(0).to(I32)


# ------------------------------------------------------------------ the plan

def plan_case(B, page, width, most_new, seed, release=True):
    g = torch.Generator().manual_seed(seed)
    most = page * width
    news = torch.randint(0, min(most, most_new) + 1, (B,), generator=g)
    lens = (torch.rand(B, generator=g, dtype=torch.float64) * (most - news + 1)).long()
    gone = torch.rand(B, generator=g) < 0.3 if release else torch.zeros(B, dtype=torch.bool)
    have = (lens + page - 1) // page
    pool = B * width + 3
    order = torch.randperm(pool, generator=g)
    table = torch.full((B, width), -9)
    held = torch.arange(width) < have[:, None]
    n = int(have.sum())
    table[held] = order[:n]
    free = torch.full((pool,), -5)
    free[:pool - n] = order[n:]
    return table, lens, news, free, torch.tensor([pool - n]), gone


def plan_run(case, page, tokens, **kw):
    table, lens, news, free, count, gone = (t.to("cuda", I32) for t in case)
    got = K.page_plan(table, lens, news, free, count, page, tokens, release=gone.bool(), **kw)
    K.check_device_error()
    return got, (table, lens, free, count)


def plan_check(got, ref):
    for g, r, name in zip(got, ref, ("table", "lens", "free", "count", "cu", "positions", "slots")):
        g = g.cpu()
        r = torch.tensor(r).to(g.dtype).reshape(g.shape)
        assert torch.equal(g, r), name


@pytest.mark.parametrize("B,page,width,new,extra", [
    (1, 16, 4, 1, 0), (1, 1, 300, 300, 3), (5, 16, 7, 40, 0), (37, 17, 9, 1, 12), (64, 64, 40, 500, 1),
    (300, 1, 20, 9, 0), (1024, 32, 3, 2, 0), (1025, 8, 2, 16, 5), (2500, 100, 1, 5, 0), (3, 8, 700, 5600, 0)])
def test_plan(B, page, width, new, extra):
    case = plan_case(B, page, width, new, B + page)
    tokens = int(case[2].sum()) + extra
    ref = C.page_plan(*case[:4], int(case[4]), page, tokens, case[5])
    got, before = plan_run(case, page, tokens)
    plan_check(got, ref)
    assert all(torch.equal(b.cpu().long(), c) for b, c in zip(before, (case[0], case[1], case[3], case[4])))
    got, state = plan_run(case, page, tokens, in_place=True)
    plan_check(got, ref)
    assert all(a.data_ptr() == b.data_ptr() for a, b in zip(got, state))


@pytest.mark.parametrize("B,page,width,new", [(4096, 16, 3, 2), (4097, 16, 3, 2), (9000, 8, 2, 16)])
def test_plan_of_many_slots(B, page, width, new):
    """At and past the slots whose sums a block holds."""
    test_plan(B, page, width, new, 2)


def test_plan_steps_follow_one_another():
    """A batch served for a while, in place, with slots given back and filled again."""
    g = torch.Generator().manual_seed(7)
    B, page, width, pool = 9, 4, 6, 60
    state = [torch.zeros(B, width).tolist(), [0] * B, list(range(pool)), pool]
    dev = [i32([[0] * width] * B), i32([0] * B), i32(list(range(pool))), i32([pool])]
    for step in range(40):
        gone = [torch.rand((), generator=g).item() < 0.15 for _ in range(B)]
        news = [int(torch.randint(0, 4, (), generator=g)) for _ in range(B)]
        for i in range(B):
            if (0 if gone[i] else state[1][i]) + news[i] > page * width:
                gone[i] = True
        ref = C.page_plan(state[0], state[1], news, state[2], state[3], page, 40, gone)
        got = K.page_plan(*dev[:2], i32(news), *dev[2:], page, 40, release=torch.tensor(gone).cuda(),
                          in_place=True)
        plan_check(got, ref)
        state = list(ref[:4])
    K.check_device_error()
    used = [p for i in range(B) for p in state[0][i][:-(-state[1][i] // page)]]
    assert sorted(used + state[2][:state[3]]) == list(range(pool))   # no page lost or held twice


@pytest.mark.parametrize("B,page,width,new", [(16, 16, 8, 30), (64, 16, 20, 200), (1100, 8, 3, 5)])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan_captured_into_a_graph(B, page, width, new, in_place):
    """Every form's launches, replayed: in place each replay goes on from the one before, with
    all slots given back and filled anew."""
    table, lens, news, free, count, gone = plan_case(B, page, width, new, 11)
    gone[:] = True
    tokens = int(news.sum()) + 7
    dev = [t.to("cuda", I32) for t in (table, lens, news, free, count)]
    rel = gone.cuda()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        K.page_plan(*dev, page, tokens, release=rel)   # (its workspace)
        K.page_plan(*(t.clone() for t in dev), page, tokens, release=rel, in_place=True)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            got = K.page_plan(*dev, page, tokens, release=rel, in_place=in_place)
        state = table, lens, free, int(count)
        for _ in range(3):
            graph.replay()
            ref = C.page_plan(state[0], state[1], news, state[2], state[3], page, tokens, gone)
            if in_place:
                state = ref[:4]
            stream.synchronize()
            plan_check(got, ref)
    K.check_device_error()


@pytest.mark.parametrize("fault,error", [
    ("long", "PAGE_TABLE"), ("negative", "PAGE_TABLE"), ("held", "PAGE_TABLE"), ("rows", "PAGE_TABLE"),
    ("count", "PAGE_TABLE"), ("pool", "OUT_OF_PAGES")])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan_refuses_as_a_whole(fault, error, in_place):
    table, lens, news, free, count, gone = plan_case(20, 8, 6, 10, 3, release=False)
    tokens = int(news.sum())
    lens[4], news[4] = 3, 2
    tokens = int(news.sum())
    if fault == "long":
        news[4] = 46
    elif fault == "negative":
        news[4] = -1
    elif fault == "held":
        lens[4] = 49
    elif fault == "rows":
        tokens -= 1
    elif fault == "count":
        count[0] = len(free) + 1
    else:
        need = sum(-(-(a + b) // 8) - -(-a // 8) for a, b in zip(lens.tolist(), news.tolist()))
        count[0] = need - 1
    dev = [t.to("cuda", I32) for t in (table, lens, news, free, count)]
    got = K.page_plan(*dev, 8, tokens, in_place=in_place)
    with pytest.raises(K.KdaError, match=error):
        K.check_device_error()
    for g, r in zip(got, (table, lens, free, count)):
        assert torch.equal(g.cpu().long(), r)
    assert not got[4].any() and not got[5].any() and (got[6] == -1).all()


@pytest.mark.parametrize("B", [70, 1100])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("fault", ["rows", "pool", "held"])
def test_large_plan_refuses_as_a_whole(fault, in_place, B):
    """Likewise where several blocks fill the tables."""
    table, lens, news, free, count, gone = plan_case(B, 16, 200, 300, 4)
    lens[B - 1], news[B - 1], gone[B - 1] = 5, 12, False
    tokens = int(news.sum()) - (fault == "rows")
    if fault == "pool":
        count[0] = 0
        gone[:] = False
    elif fault == "held":
        lens[B - 1] = 16 * 200 + 1
    dev = [t.to("cuda", I32) for t in (table, lens, news, free, count)]
    got = K.page_plan(*dev, 16, tokens, release=gone.cuda(), in_place=in_place)
    with pytest.raises(K.KdaError, match="OUT_OF_PAGES" if fault == "pool" else "PAGE_TABLE"):
        K.check_device_error()
    for g, r in zip(got, (table, lens, free, count)):
        assert torch.equal(g.cpu().long(), r)
    assert not got[4].any() and not got[5].any() and (got[6] == -1).all()


def test_plan_without_slots_or_tokens():
    got = K.page_plan(i32([]).view(0, 4), i32([]), i32([]), i32([3, 1]), i32([2]), 16, 3)
    assert got[4].tolist() == [0] and got[6].tolist() == [-1] * 3 and got[2].tolist() == [3, 1]
    got = K.page_plan(i32([[1], [2]]), i32([5, 0]), i32([0, 0]), i32([]), i32([0]), 16, 0,
                      release=torch.tensor([False, True]).cuda())
    K.check_device_error()
    assert got[4].tolist() == [0, 0, 0] and got[0].tolist() == [[1], [2]] and got[1].tolist() == [5, 0]


# ------------------------------------------------------- norms and rotation

HEADS = [
    # T, Hq, Hk, D, R, pairs, fused, farthest position
    (1, 1, 0, 128, 128, False, False, 0),
    (1, 32, 8, 128, 128, False, True, 1 << 20),
    (7, 3, 1, 64, 64, True, True, 100),
    (130, 5, 2, 128, 64, False, True, 5000),
    (65, 8, 1, 256, 256, True, False, 1 << 24),
    (33, 1, 1, 256, 96, False, True, 77),
    (300, 2, 1, 64, 16, False, True, 300),
    (9, 70, 3, 128, 112, True, True, 40000),
    (20, 4, 4, 64, 0, False, True, 0),
    (513, 1, 0, 64, 48, False, False, 10),
]


def heads_case(T, Hq, Hk, D, R, pairs, fused, far, weights=True, seed=0):
    r = make(seed + T + D + R)
    H = Hq + 2 * Hk
    x = r(T, H * D + 8) if fused else r(T, H * D)
    q = x[:, :Hq * D].unflatten(1, (Hq, D))
    k = x[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D)) if Hk else None
    if not fused:
        q, k = q.contiguous(), None if k is None else k.contiguous()
    w = [1 + 0.3 * r(D, dtype=F32) if weights else None for _ in range(2)]
    g = torch.Generator().manual_seed(T)
    pos = torch.randint(0, far + 1, (T,), generator=g).to("cuda", I32) if R else None
    freq = (10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / max(R, 1))).float().cuda() if R else None
    return r, q, k, w, freq, pos


@pytest.mark.parametrize("weights", [True, False])
@pytest.mark.parametrize("T,Hq,Hk,D,R,pairs,fused,far", HEADS)
def test_heads(T, Hq, Hk, D, R, pairs, fused, far, weights):
    _, q, k, w, freq, pos = heads_case(T, Hq, Hk, D, R, pairs, fused, far, weights)
    nan = torch.full((T, 2, (Hq + Hk) * D), float("nan"), dtype=BF16, device="cuda")
    qo = nan[:, 1, :Hq * D].unflatten(1, (Hq, D))
    ko = nan[:, 1, Hq * D:].unflatten(1, (Hk, D)) if Hk else None
    K.qk_norm_rope(q, k, *w, freq, pos, interleaved=pairs, q_out=qo, k_out=ko)
    assert torch.isnan(nan[:, 0]).all()
    close(qo, *C.norm_rope(q, w[0], freq, pos, interleaved=pairs), "q")
    if Hk:
        close(ko, *C.norm_rope(k, w[1], freq, pos, interleaved=pairs), "k")
    # made here, and in place, the same bits
    a = K.qk_norm_rope(q, k, *w, freq, pos, interleaved=pairs)
    assert torch.equal(a[0], qo) and (k is None) == (a[1] is None)
    K.qk_norm_rope(q, k, *w, freq, pos, interleaved=pairs, q_out=q, k_out=k)
    assert torch.equal(q, qo) and (k is None or torch.equal(k, ko))


@pytest.mark.parametrize("d32", [True, False])
@pytest.mark.parametrize("T,Hq,Hk,D,R,pairs,fused,far", HEADS)
def test_heads_gradient(T, Hq, Hk, D, R, pairs, fused, far, d32):
    r, q, k, w, freq, pos = heads_case(T, Hq, Hk, D, R, pairs, fused, far)
    dtype = F32 if d32 else BF16
    dy = r(T, (Hq + Hk) * D + 8, dtype=dtype)
    dqo = dy[:, :Hq * D].unflatten(1, (Hq, D))
    dko = dy[:, Hq * D:-8].unflatten(1, (Hk, D)) if Hk else None
    dx = torch.full((T, (Hq + Hk + 1) * D), float("nan"), dtype=BF16, device="cuda")
    dq = dx[:, :Hq * D].unflatten(1, (Hq, D))
    dk = dx[:, Hq * D:-D].unflatten(1, (Hk, D)) if Hk else None
    kw = dict(interleaved=pairs, eps=1e-5)
    got = K.qk_norm_rope_backward(q, k, dqo, dko, *w, freq, pos, dq=dq, dk=dk, **kw)
    assert torch.isnan(dx[:, -D:]).all()
    for x, dyo, wi, d, dw, name in ((q, dqo, w[0], got[0], got[2], "q"), (k, dko, w[1], got[1], got[3], "k")):
        if x is None:
            assert d is None and dw is None
            continue
        rx, rw = C.norm_rope_backward(x, dyo, wi, freq, pos, 1e-5, pairs)
        close(d, *rx, "d" + name)
        close(dw, *rw, f"d{name}_weight")
    again = K.qk_norm_rope_backward(q, k, dqo, dko, *w, freq, pos, **kw)
    assert all(a is None and b is None or torch.equal(a, b) for a, b in zip(got, again)), "other bits"
    bare = K.qk_norm_rope_backward(q, k, dqo, dko, None, None, freq, pos, **kw)
    assert bare[2] is None and bare[3] is None
    close(bare[0], *C.norm_rope_backward(q, dqo, None, freq, pos, 1e-5, pairs)[0], "dq without weights")


def test_heads_gradient_against_differences():
    """Directional derivatives of the reference's forward pass; the bound is the rounding of
    dx to bf16 (2^-8 of it, at random) and the differences' own error."""
    r, q, k, w, freq, pos = heads_case(40, 3, 2, 64, 32, False, True, 1000)
    dq, dk = r(40, 3, 64, dtype=F32), r(40, 2, 64, dtype=F32)
    got = K.qk_norm_rope_backward(q, k, dq, dk, *w, freq, pos, eps=1e-3)
    g = torch.Generator().manual_seed(3)
    for x, dy, wi, dx, dw in ((q, dq, w[0], got[0], got[2]), (k, dk, w[1], got[1], got[3])):
        xd, wd, dyd = x.cpu().double(), wi.cpu().double(), dy.cpu().double()

        def loss(a, b):
            return float((C.norm_rope(a, b, freq, pos, 1e-3)[0] * dyd).sum())

        u, e = torch.randn(xd.shape, generator=g, dtype=torch.float64), 1e-5
        diff = (loss(xd + e * u, wd) - loss(xd - e * u, wd)) / (2 * e)
        mine = dx.cpu().double() * u
        assert abs(float(mine.sum()) - diff) <= 2.0 ** -8 * float(mine.norm()) * 4 + 1e-6 * float(mine.abs().sum())
        u = torch.randn(64, generator=g, dtype=torch.float64)
        diff = (loss(xd, wd + e * u) - loss(xd, wd - e * u)) / (2 * e)
        mine = dw.cpu().double() * u
        assert abs(float(mine.sum()) - diff) <= 1e-5 * float(mine.abs().sum())


@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_heads_ends_of_the_range(eps):
    """Rows of zeros, of tiny and of huge numbers, and rows that hold an infinity or NaN, which
    keep to themselves."""
    _, q, k, w, freq, pos = heads_case(8, 4, 2, 128, 128, False, False, 100)
    q[0], q[1, 0], q[1, 1] = 0, 2.0 ** -60, 2.0 ** 58
    q[2, 1, 7], q[3, 2, 100] = math.inf, math.nan
    a, _ = K.qk_norm_rope(q, k, *w, freq, pos, eps=eps)
    ref, size = C.norm_rope(q, w[0], freq, pos, eps)
    odd = torch.zeros(8, 4, dtype=torch.bool)
    odd[2, 1] = odd[3, 2] = True
    if eps == 0:
        odd[0] = True
        assert torch.isnan(a[0]).all()
    else:
        assert not a[0].any()
    close(a.cpu()[~odd], ref[~odd], size[~odd], "q")
    assert torch.isnan(a[3, 2]).all() and torch.isnan(a.float()[2, 1]).any()


def test_heads_far_positions():
    """At position p an angle may be off by 2^-20 of a turn (up to 2^24), whatever its frequency."""
    T = 64
    pos = i32([(1 << 24) - 1 - 37 * i for i in range(T // 2)] + [-5 - 4097 * i for i in range(T // 2)])
    x = torch.zeros(T, 1, 128, dtype=BF16, device="cuda")
    x[..., :64] = 1.0   # y = cos, sin times sqrt(2)
    freq = torch.rand(64, generator=torch.Generator().manual_seed(1)).cuda()
    y, _ = K.qk_norm_rope(x, None, None, None, freq, pos, eps=0.0)
    close(y, *C.norm_rope(x, None, freq, pos, 0.0), "y")


def test_heads_without_tokens_and_batched():
    r = make(5)
    w = 1 + r(64, dtype=F32)
    q = torch.empty(0, 2, 64, dtype=BF16, device="cuda")
    a, b = K.qk_norm_rope(q, q, w, w)
    assert a.shape == q.shape and b.shape == q.shape
    dq, dk, dqw, dkw = K.qk_norm_rope_backward(q, q, q, q, w, w)
    assert not dqw.any() and not dkw.any()
    q, pos = r(3, 11, 2, 64), i32([[5 * i + j for j in range(11)] for i in range(3)])
    freq = torch.rand(32, device="cuda")
    a, _ = K.qk_norm_rope(q, None, w, None, freq, pos)
    b, _ = K.qk_norm_rope(q.view(33, 2, 64), None, w, None, freq, pos.view(-1))
    assert torch.equal(a.view(33, 2, 64), b)


# ----------------------------------------------------------- into the cache

LAYOUTS = ["page", "token", "heads first", "apart"]


def empty_cache(pages, page, H, D, layout):
    """(k_cache, v_cache, k_scale, v_scale) in one buffer or two, filled with NaN codes."""
    if layout == "page":       # keys beside values in a page
        both = torch.empty(pages, 2, page, H, D, dtype=torch.uint8, device="cuda").fill_(127)
        k, v = both[:, 0], both[:, 1]
    elif layout == "token":    # in a token
        both = torch.empty(pages, page, 2, H, D, dtype=torch.uint8, device="cuda").fill_(127)
        k, v = both[:, :, 0], both[:, :, 1]
    elif layout == "heads first":
        both = torch.empty(pages, 2, H, page, D, dtype=torch.uint8, device="cuda").fill_(127)
        k, v = both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2)
    else:
        k, v = (torch.empty(pages, page, H, D, dtype=torch.uint8, device="cuda").fill_(127) for _ in range(2))
    scales = torch.full((pages, 2, H), float("nan"), device="cuda")
    return k.view(F8), v.view(F8), scales[:, 0], scales[:, 1]


def deal(lens, page, spare, seed):
    need = [-(-n // page) for n in lens]
    order = torch.randperm(sum(need) + spare, generator=torch.Generator().manual_seed(seed))
    table = torch.full((len(lens), max(1, *need)), -1, dtype=I32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    return table, sum(need) + spare


def same_cache(dev, ref):
    for (codes, scale), (rc, rs), name in zip(((dev[0], dev[2]), (dev[1], dev[3])), ref, "kv"):
        codes, scale = codes.cpu().double(), scale.cpu().double()
        assert torch.equal(torch.isnan(codes), torch.isnan(rc)), name
        assert torch.equal(codes.nan_to_num(0), rc.nan_to_num(0)), name
        assert torch.equal(scale.nan_to_num(-1), rs.nan_to_num(-1)), name + " scale"


APPEND = [
    # rounds of new tokens for each slot, H, D, page
    ([[1]], 1, 128, 16),
    ([[5, 0, 40, 1]], 2, 64, 16),
    ([[3, 20, 0], [14, 1, 7], [1, 1, 1]], 3, 128, 8),
    ([[130, 1], [1, 300], [70, 0]], 2, 128, 64),
    ([[257, 12]], 1, 64, 128),
    ([[9, 4], [1, 1], [1, 1], [6, 0]], 5, 128, 1),
    ([[33, 90], [50, 17]], 2, 64, 17),
    ([[600], [500]], 1, 128, 300),
    ([[2] * 40, [1] * 40], 1, 64, 32),
]


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("rounds,H,D,page", APPEND)
def test_append(rounds, H, D, page, layout):
    B = len(rounds[0])
    ends = [sum(r[i] for r in rounds) for i in range(B)]
    table, pages = deal(ends, page, 2, B + page)
    dev = empty_cache(pages, page, H, D, layout)
    ref = [(c.cpu().double(), s.cpu().double()) for c, s in ((dev[0], dev[2]), (dev[1], dev[3]))]
    r, lens = make(D + page), [0] * B
    for n, new in enumerate(rounds):
        lens = [a + b for a, b in zip(lens, new)]
        T = sum(new)
        x = r(T + 3, 3, H, D, scale=3.0 ** n)      # later tokens are larger: scales grow
        x *= torch.exp2(torch.randint(-3, 3, (T + 3, 1, 1, 1), device="cuda").float())
        x[T:] = float("nan")                       # rows behind the last slot
        step = new == [1] * B
        cu = None if step else cu_of(new)
        k, v = (x[:T, i] if step else x[:, i] for i in (1, 2))
        K.paged_append_fp8(k, v, *dev, table.cuda(), i32(lens), None if step else cu.cuda())
        K.check_device_error()
        for x, (codes, scale) in zip((k, v), ref):
            C.append(x, codes, scale, table, lens, cu)
        same_cache(dev, ref)


@pytest.mark.parametrize("H,D,layout", [(8, 64, "page"), (1, 64, "heads first"), (3, 128, "heads first"),
                                        (17, 128, "page")])
def test_append_pages_of_one(H, D, layout):
    """Slots more than a warp's lanes, some without new tokens; infinities and NaN; a bad page."""
    B = 75
    g = torch.Generator().manual_seed(H)
    old = torch.randint(0, 4, (B,), generator=g).tolist()
    new = torch.randint(0, 6, (B,), generator=g).tolist()
    new[-1] = 0
    lens = [a + b for a, b in zip(old, new)]
    table, pages = deal(lens, 1, 2, H)
    dev = empty_cache(pages, 1, H, D, layout)
    ref = [(c.cpu().double(), s.cpu().double()) for c, s in ((dev[0], dev[2]), (dev[1], dev[3]))]
    T = sum(new)
    x = make(H + D)(T + 9, 2, H, D)
    x[5, 0, 0, 3], x[6, 1, H - 1, 0], x[7] = math.inf, math.nan, -math.inf
    x[T:] = float("nan")
    k, v, cu = x[:, 0], x[:, 1], cu_of(new)
    K.paged_append_fp8(k, v, *dev, table.cuda(), i32(lens), cu.cuda())
    K.check_device_error()
    for y, (codes, scale) in zip((k, v), ref):
        C.append(y, codes, scale, table, lens, cu)
    same_cache(dev, ref)
    bad, at = table.clone(), max(i for i in range(B) if new[i])
    bad[at, lens[at] - 1] = pages
    again = empty_cache(pages, 1, H, D, layout)
    K.paged_append_fp8(k, v, *again, bad.cuda(), i32(lens), cu.cuda())
    with pytest.raises(K.KdaError, match="PAGE_TABLE"):
        K.check_device_error()
    page = int(table[at, lens[at] - 1])
    for a, b in zip(again, dev):
        a, b = (t.view(torch.uint8) if t.dtype == F8 else t.view(I32) for t in (a, b))
        keep = torch.arange(pages, device="cuda") != page
        assert torch.equal(a[keep], b[keep])
    assert torch.isnan(again[2][page]).all()


def test_append_ends_of_the_range():
    """Zeros, the smallest and the largest bf16 numbers, infinities and NaN, values at the
    borders of two scales, and scales that a caller has set."""
    big, tiny = torch.finfo(BF16).max, 2.0 ** -133
    rows = [[0.0, 0.0], [tiny, -tiny], [big, -big], [math.inf, 3.0], [-math.inf, math.nan], [448.0, 1.0],
            [450.0, 1.0], [1.75, 1.0], [1.7578125, 1.0], [2.0 ** -126, 0.0], [448.0, 17.0], [448.0, 2.0 ** -9],
            [448.0, 2.0 ** -10], [448.0, 1.5 * 2.0 ** -9]]
    x = torch.zeros(len(rows), 1, 64)
    x[:, 0, :2] = torch.tensor(rows)
    x = x.to(BF16).cuda()
    table = torch.arange(len(rows), dtype=I32)[:, None]
    for first in (0, 1):
        dev = empty_cache(len(rows), 4, 1, 64, "page")
        for codes, scale in ((dev[0], dev[2]), (dev[1], dev[3])):
            codes.view(torch.uint8).copy_(torch.randint(0, 126, codes.shape, device="cuda", dtype=torch.uint8))
            scale.copy_(torch.exp2(torch.arange(len(rows), device="cuda").float() - 7)[:, None])
        dev[3][3:6] = 0.3
        ref = [(c.cpu().double(), s.cpu().double()) for c, s in ((dev[0], dev[2]), (dev[1], dev[3]))]
        lens = [first + 1] * len(rows)
        K.paged_append_fp8(x, x, *dev, table.cuda(), i32(lens))
        K.check_device_error()
        for codes, scale in ref:
            C.append(x, codes, scale, table, lens)
        if first:   # a scale of 0.3 in fp32: its reciprocal's rounding may move a tie
            keep = [i for i in range(len(rows)) if i not in (3, 4, 5)]
            assert (dev[3][3:6].cpu().double() == ref[1][1][3:6]).all()
            got = dev[1].cpu().double()[3:6]
            want = ref[1][0][3:6]
            assert torch.equal(torch.isnan(got), torch.isnan(want))
            # one step: 2^-3 of a number 2^e, and 2^-9 between the smallest (below 2^-6)
            off = (got - want).nan_to_num(0).abs()
            assert bool((off <= (2.0 ** -3 * want.nan_to_num(0).abs()).clamp(min=2.0 ** -9)).all())
            dev = [t[keep] if t.dtype == F32 else t.view(torch.uint8)[keep].view(F8) for t in dev]
            ref = [(c[keep], s[keep]) for c, s in ref]
        same_cache(dev, ref)


def test_append_bad_lengths_pages_and_cu():
    r = make(2)
    H, D, page = 2, 64, 8
    x = r(30, H, D)
    table, pages = deal([20, 20, 20], page, 1, 0)

    def go(cu, lens, table):
        dev = empty_cache(pages, page, H, D, "page")
        K.paged_append_fp8(x, x, *dev, table.cuda(), i32(lens), i32(cu))
        return dev

    good = go([0, 10, 20, 30], [20, 20, 20], table)
    K.check_device_error()

    def untouched(dev, slots, pages_of=lambda i: table[i].tolist()):
        for i in range(3):
            for p in pages_of(i):
                same = torch.equal(dev[0][p].view(torch.uint8), good[0][p].view(torch.uint8))
                blank = (dev[0][p].view(torch.uint8) == 127).all() and torch.isnan(dev[2][p]).all()
                assert blank if i in slots else same, (i, p)

    for lens in ([20, -1, 20], [20, 9, 20], [20, 1000, 20]):
        dev = go([0, 10, 20, 30], lens, table)
        with pytest.raises(K.KdaError, match="PAGE_TABLE"):
            K.check_device_error()
        untouched(dev, [1])
    for bad in (-1, pages, 1 << 30):
        t = table.clone()
        t[1] = bad
        dev = go([0, 10, 20, 30], [20, 20, 20], t)
        with pytest.raises(K.KdaError, match="PAGE_TABLE"):
            K.check_device_error()
        untouched(dev, [1])
    for cu in ([0, 10, 20, 31], [5, 10, 20, 30], [0, 20, 10, 30], [-4, 10, 20, 30], [0, 1 << 30, 20, 30]):
        go(cu, [20, 20, 20], table)
        with pytest.raises(K.KdaError, match="CU_SEQLENS"):
            K.check_device_error()


def test_append_and_decode_offsets_past_32_bits():
    """Pages that lie more than 2^32 bytes into the cache."""
    page, H, D, pages = 128, 8, 128, 40000          # 10.5 GB
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 11 GB")
    both = torch.empty(pages, 2, page, H, D, dtype=F8, device="cuda")
    scales = torch.empty(2, pages, H, device="cuda")
    dev = (both[:, 0], both[:, 1], scales[0], scales[1])
    r, table = make(6), i32([[39999, 0, 39998, 20000]])
    k, v, q = r(470, H, D), r(470, H, D), r(1, 16, D)
    K.paged_append_fp8(k, v, *dev, table, i32([470]), i32([0, 470]))
    o, l = K.paged_decode_fp8(q, *dev, table, i32([470]))
    K.check_device_error()
    ids = table[0].long()
    small = [t[ids] if t.dtype == F32 else t.view(torch.uint8)[ids].view(F8) for t in dev]
    ref = [(torch.zeros(4, page, H, D, dtype=torch.float64), torch.zeros(4, H, dtype=torch.float64)) for _ in "kv"]
    at = torch.arange(4, dtype=I32)[None]
    for x, (codes, scale) in zip((k, v), ref):
        C.append(x, codes, scale, at, [470], [0, 470])
    for t, (codes, scale) in zip(small[:2], ref):
        assert torch.equal(t.cpu().double().flatten(0, 1)[:470], codes.flatten(0, 1)[:470])
    attention_close(o, l, q, *small, at, [470])


# -------------------------------------------------------------- the attention

def cache_case(lens, Hq, Hkv, D, page, layout="page", seed=0, spread=3):
    """Random numbers at random scales; NaN in every row that no sequence holds."""
    table, pages = deal(lens, page, 3, seed)
    r = make(seed + Hq + D + page)
    dev = empty_cache(pages, page, Hkv, D, layout)
    g = torch.Generator(device="cuda").manual_seed(seed)
    for s in dev[2:]:
        s.copy_(torch.exp2(torch.randint(-spread, spread + 1, s.shape, generator=g, device="cuda").float()))
    used = torch.zeros(pages, page, dtype=torch.bool)
    for i, n in enumerate(lens):
        for t in range(0, n, page):
            used[int(table[i, t // page]), :min(page, n - t)] = True
    for c, s in zip(dev[:2], dev[2:]):
        x = r(pages, page, Hkv, D, dtype=F32) / s[:, None, :, None]
        x[~used.cuda()] = float("nan")
        c.view(torch.uint8).copy_(x.to(F8).view(torch.uint8))
    return (r(len(lens), Hq, D), *dev, table.cuda(), i32(lens))


def attention_close(out, lse, q, kc, vc, ks, vs, table, lens, scale=None):
    ro, rl, size, reach, floor = C.paged_attention(q, kc, vc, ks, vs, table, lens, scale)
    # weights p carry the error of their score, at most 2^-18 of sum |q||k|; below 2^-16 of the
    # largest (times the values' scales) they keep less than 16 bits: the last of four terms of
    # e4m3, 32 times finer each and starting from 2^8, steps by 2^-9 / 32^3 / 2^8 = 2^-32, and half
    # of that is lost (`close` allows 2^-12 of what it is given)
    close(out, ro, size * (1 + 2.0 ** -6 * reach[..., None]) + 2.0 ** (12 - 33) * floor, "out")
    lse = lse.cpu().double()
    empty = torch.isinf(rl)
    assert torch.equal(torch.isinf(lse) & (lse < 0), empty)
    err = (lse - rl)[~empty].abs() - 2.0 ** -18 * (1 + reach + rl.abs())[~empty]
    assert err.numel() == 0 or float(err.max()) <= 0, "lse"


PAGED = [
    # lens, Hq, Hkv, D, page, layout
    ([1], 1, 1, 128, 16, "page"),
    ([0, 1, 15, 16, 17, 1000], 8, 2, 128, 16, "token"),
    ([63, 64, 65, 128, 129], 4, 4, 64, 64, "apart"),
    ([127, 128, 129, 255, 257, 0, 511], 8, 1, 128, 32, "heads first"),
    ([700], 32, 8, 128, 1, "page"),
    ([100, 3, 0, 0, 517], 12, 4, 128, 17, "heads first"),
    ([2049, 5], 16, 1, 128, 100, "token"),
    ([300, 777], 20, 1, 64, 32, "page"),
    ([90], 64, 1, 128, 128, "heads first"),
    ([1200] * 3, 80, 2, 128, 64, "page"),
    ([17] * 40, 6, 2, 64, 8, "apart"),
    ([1, 400], 5, 1, 64, 300, "heads first"),
]


@pytest.mark.parametrize("lens,Hq,Hkv,D,page,layout", PAGED)
def test_decode(lens, Hq, Hkv, D, page, layout):
    case = cache_case(lens, Hq, Hkv, D, page, layout)
    out = torch.full_like(case[0], float("nan"))
    lse = torch.full((len(lens), Hq), float("nan"), device="cuda")
    o, l = K.paged_decode_fp8(*case, out=out, lse=lse)
    K.check_device_error()
    attention_close(o, l, *case[:6], lens)
    o2, l2 = K.paged_decode_fp8(*case)
    assert torch.equal(o, o2) and torch.equal(l, l2), "not the same bits again"


def test_decode_long_and_ragged():
    lens = [40000, 1, 0, 9000, 123]
    case = cache_case(lens, 16, 4, 128, 32)
    o, l = K.paged_decode_fp8(*case)
    K.check_device_error()
    attention_close(o, l, *case[:6], lens)


@pytest.mark.parametrize("lens,Hq,Hkv,D,page,scale", [
    ([20000], 7, 1, 128, 17, None), ([20000], 16, 1, 64, 32, None), ([30, 0, 31000, 500], 12, 1, 128, 64, None),
    ([17000, 9], 2, 2, 64, 100, 4.0), ([25000], 24, 1, 128, 8, 40.0), ([19000], 8, 1, 128, 16, -1000.0)])
def test_decode_joins_in_groups(lens, Hq, Hkv, D, page, scale):
    """Few sequences, cut into so many pieces that they are joined in two steps; with a large
    scale most pieces' weights vanish."""
    case = cache_case(lens, Hq, Hkv, D, page, "heads first", seed=6, spread=1)
    o, l = K.paged_decode_fp8(*case, scale=scale)
    K.check_device_error()
    attention_close(o, l, *case[:6], lens, *([] if scale is None else [scale]))
    for _ in range(3):
        o2, l2 = K.paged_decode_fp8(*case, scale=scale)
        assert torch.equal(o, o2) and torch.equal(l, l2)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("scale", [1.0, 4.0, -0.5, 0.0])
def test_decode_scores_far_apart(scale, D):
    """Scores of hundreds: the running maximum moves and most weights vanish."""
    lens = [5, 400, 3000]
    case = cache_case(lens, 8, 2, D, 16, seed=2, spread=1)
    o, l = K.paged_decode_fp8(*case, scale=scale)
    attention_close(o, l, *case[:6], lens, scale)


def test_decode_scales_far_apart():
    """Pages of values 2^-126 to 2^60 beside one another; pages of zeros, whose scale is
    2^-126; scales that are no powers of two."""
    lens = [150, 600, 70]
    q, kc, vc, ks, vs, table, n = cache_case(lens, 8, 2, 128, 16, seed=4)
    g = torch.Generator(device="cuda").manual_seed(1)
    for tag in ("tiny", "wide", "odd", "zero"):
        vs.copy_(torch.exp2(torch.randint(-60, 61, vs.shape, generator=g, device="cuda").float()))
        if tag == "tiny":
            vs.fill_(2.0 ** -100)
        elif tag == "odd":
            vs.copy_(torch.rand(vs.shape, generator=g, device="cuda") + 0.01)
            ks.copy_(torch.rand(ks.shape, generator=g, device="cuda") + 0.01)
        elif tag == "zero":
            vs.fill_(2.0 ** -126)
            vs[::2] = 1.0
        o, l = K.paged_decode_fp8(q, kc, vc, ks, vs, table, n)
        attention_close(o, l, q, kc, vc, ks, vs, table, lens)
    vc.view(torch.uint8).zero_()
    vs.fill_(2.0 ** -126)
    o, l = K.paged_decode_fp8(q, kc, vc, ks, vs, table, n)
    assert not o.any()
    attention_close(o, l, q, kc, vc, ks, vs, table, lens)


@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** 60])
def test_decode_queries_far_apart(size):
    """Tiny and huge queries (the scale brings the scores back), and a row of zeros."""
    lens = [200, 33]
    q, kc, vc, ks, vs, table, n = cache_case(lens, 8, 2, 128, 16, seed=6)
    q = (q.float() * size).to(BF16)
    q[0, 3] = 0
    o, l = K.paged_decode_fp8(q, kc, vc, ks, vs, table, n, scale=1 / (size * 12))
    attention_close(o, l, q, kc, vc, ks, vs, table, lens, 1 / (size * 12))


def test_decode_non_finite_numbers_keep_to_their_rows():
    lens = [300, 40]
    q, kc, vc, ks, vs, table, n = cache_case(lens, 8, 2, 128, 16, seed=8)
    o, l = K.paged_decode_fp8(q, kc, vc, ks, vs, table, n)
    kv = kc.view(torch.uint8)
    kv[int(table[0, 3]), 5, 1, 9] = 127          # a NaN among the keys of head 1
    q[1, 2, 3] = math.nan
    q[1, 6, 0] = math.inf
    o2, l2 = K.paged_decode_fp8(q, kc, vc, ks, vs, table, n)
    odd = torch.zeros(2, 8, dtype=torch.bool)
    odd[0, 4:] = True
    odd[1, 2] = odd[1, 6] = True
    assert torch.isnan(o2[odd.cuda()]).all() and torch.isnan(l2[odd.cuda()]).all()
    assert torch.equal(o2[~odd.cuda()], o[~odd.cuda()]) and torch.equal(l2[~odd.cuda()], l[~odd.cuda()])
    kv[int(table[0, 3]), 5, 1, 9] = 0
    vc.view(torch.uint8)[int(table[0, 0]), 2, 0, 77] = 127   # among the values: that channel
    o3, l3 = K.paged_decode_fp8(q, kc, vc, ks, vs, table, n)
    assert torch.isnan(o3[0, :4, 77]).all() and torch.isfinite(o3[0, :4, :77]).all()
    assert torch.isfinite(l3[0]).all()


@pytest.mark.parametrize("page", [16, 17])
def test_decode_strides_of_no_pattern(page):
    """Rows, heads and pages a multiple of 16 bytes apart, but of nothing else."""
    lens, pages, Hkv, D = [200, 75], 20, 3, 64
    q, kc, vc, ks, vs, table, n = cache_case(lens, 6, Hkv, D, page)
    ref = K.paged_decode_fp8(q, kc, vc, ks, vs, table, n)
    pages = kc.shape[0]
    steps = (Hkv * (page * 80 + 48) + 16, 80, page * 80 + 48)   # page, token, head
    apart = []
    for c in (kc, vc):
        t = torch.empty(pages * steps[0], dtype=torch.uint8, device="cuda").fill_(127)
        t = t.as_strided(c.shape, (*steps, 1))
        t.copy_(c.view(torch.uint8))
        apart.append(t.view(F8))
    wide = [torch.full((pages, 2 * Hkv + 1), float("nan"), device="cuda")[:, :Hkv] for _ in "kv"]
    for w, s in zip(wide, (ks, vs)):
        w.copy_(s)
    got = K.paged_decode_fp8(q, *apart, *wide, table, n)
    K.check_device_error()
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


def test_decode_longest_cache():
    """2^31 - 4096 tokens, one page again and again: the attention over that page. A thread adds
    up 2^31 / 152 / 256 = 55000 weights of about the same size in fp32, so each sum is within
    55000 * 2^-24 = 2^-8.2 of itself, and the output within twice that."""
    q, kc, vc, ks, vs, table, n = cache_case([4096], 4, 1, 64, 4096, seed=3)
    ref, l = K.paged_decode_fp8(q, kc, vc, ks, vs, table, n)
    reps = (1 << 31) // 4096 - 1
    o, m = K.paged_decode_fp8(q, kc, vc, ks, vs, table[:, :1].expand(1, reps).contiguous(), i32([reps * 4096]))
    K.check_device_error()
    assert ((m - l - math.log(reps)).abs() <= 2.0 ** -8).all()
    at = int(table[0, 0])
    assert ((o.float() - ref.float()).abs() <= 2.0 ** -7 * vc[at].float().abs().max() * vs[at].max()).all()


@pytest.mark.parametrize("page", [16, 17])
@pytest.mark.parametrize("lens,tile", [([300], 0), ([40000, 9, 3000], 2), ([40000, 9, 3000], 3)])
def test_decode_wait_runs_out_then_clean_call(lens, tile, page):
    """(A share of the second batch is four or five tiles of 128 tokens.)"""
    runs_out_then_clean(cache_case(lens, 16, 2, 128, page), tile)


@pytest.mark.parametrize("Hq,D,page", [(32, 128, 16), (32, 128, 17), (16, 64, 16), (32, 64, 17)])
def test_decode_wait_runs_out_in_other_shapes(Hq, D, page):
    runs_out_then_clean(cache_case([40000, 9, 3000], Hq, 2, D, page), 2)


def runs_out_then_clean(case, tile):
    ref = K.paged_decode_fp8(*case)
    K.check_device_error()
    assert K.kda_test_stall_paged_fp8(tile) == 0
    try:
        K.paged_decode_fp8(*case)
        with pytest.raises(K.KdaError, match="TIMEOUT"):
            K.check_device_error()
    finally:
        assert K.kda_test_stall_paged_fp8(-1) == 0
    K.check_device_error()
    for _ in range(2):   # the counters of the joins are right again
        got = K.paged_decode_fp8(*case)
        K.check_device_error()
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


def test_decode_same_bits_from_cold_caches():
    """Many calls, each with the caches of the GPU emptied first."""
    case = cache_case([7000, 350, 2, 12000], 16, 2, 128, 64, layout="heads first")
    big = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    ref = K.paged_decode_fp8(*case)
    for i in range(40):
        big.fill_(i)
        got = K.paged_decode_fp8(*case)
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1]), i


def test_decode_bad_tables_are_reported():
    lens = [50, 20, 40]
    q, kc, vc, ks, vs, table, n = cache_case(lens, 8, 2, 128, 16)
    for c in (kc, vc):   # (a bad page is read as page 0: nothing there is NaN)
        c.view(torch.uint8).bitwise_and_(0xbf)
    o, l = K.paged_decode_fp8(q, kc, vc, ks, vs, table, n)
    for bad_table, bad_len in ((kc.shape[0], None), (-5, None), (None, -1), (None, 10 ** 6)):
        t2, n2 = table.clone(), n.clone()
        if bad_table is not None:
            t2[1, 1] = bad_table
        else:
            n2[1] = bad_len
        o2, l2 = K.paged_decode_fp8(q, kc, vc, ks, vs, t2, n2)
        with pytest.raises(K.KdaError, match="PAGE_TABLE"):
            K.check_device_error()
        for i in (0, 2):
            assert torch.equal(o2[i], o[i]) and torch.equal(l2[i], l[i])
    K.paged_decode_fp8(q, kc, vc, ks, vs, table, n)
    K.check_device_error()


# ----------------------------------------------- together, streams and graphs

def serve_state(B, Hq, Hkv, D, page, width, seed):
    r = make(seed)
    pages = B * width
    return {"table": torch.zeros(B, width, dtype=I32, device="cuda"), "lens": i32([0] * B),
            "free": torch.arange(pages, dtype=I32, device="cuda"), "count": i32([pages]),
            "cache": empty_cache(pages, page, Hkv, D, "page"), "w": [1 + 0.2 * r(D, dtype=F32) for _ in "qk"],
            "freq": (10000.0 ** (-torch.arange(0, D, 2) / D)).float().cuda(), "page": page}


def serve(s, x, new, Hq, Hkv, release=None):
    """One call of each operator: x [T, (Hq + 2 Hkv) D] are the new tokens of all slots."""
    T, D = x.shape[0], s["w"][0].numel()
    _, _, _, _, cu, pos, slots = K.page_plan(s["table"], s["lens"], new, s["free"], s["count"], s["page"], T,
                                             release=release, in_place=True)
    q, k, v = (t.unflatten(1, (-1, D)) for t in x.split([Hq * D, Hkv * D, Hkv * D], 1))
    q, k = K.qk_norm_rope(q, k, *s["w"], s["freq"], pos)
    K.paged_append_fp8(k, v, *s["cache"], s["table"], s["lens"], cu)
    last = (cu[1:] - 1).clamp(min=0).long()
    o, l = K.paged_decode_fp8(q[last].contiguous(), *s["cache"], s["table"], s["lens"])
    return o, l, q, k, slots


@pytest.mark.parametrize("D,page", [(64, 16), (128, 64)])
def test_operators_together(D, page):
    """Prompts, then tokens, with a slot given to a new prompt: the attention of every last
    token against plain attention over all the keys and values so far. A cached number is off
    by at most 2^-4 of itself (and 2^-10 of its page's scale, at most 2^-18 of the page's
    largest); twice that, when its page was scaled down."""
    Hq, Hkv, B = 8, 2, 3
    s, r = serve_state(B, Hq, Hkv, D, page, 12, 1), make(3)
    plain = [([], []) for _ in range(B)]
    for n, new in enumerate([[70, 3, 0], [1, 1, 40], [1, 1, 1], [30, 0, 1], [0, 1, 1]]):
        gone = [n == 3 and i == 0 for i in range(B)]
        x = r(sum(new) + 2, (Hq + 2 * Hkv) * D)
        o, l, q, k, slots = serve(s, x, i32(new), Hq, Hkv, torch.tensor(gone).cuda())
        K.check_device_error()
        assert (slots[sum(new):] == -1).all()
        v, at = x[:, (Hq + Hkv) * D:].unflatten(1, (Hkv, D)), 0
        for i in range(B):
            if gone[i]:
                plain[i] = ([], [])
            plain[i][0].extend(k[at:at + new[i]].double().cpu())
            plain[i][1].extend(v[at:at + new[i]].double().cpu())
            # the slots are where the cache has them
            for j in range(new[i]):
                p, row = divmod(int(slots[at + j]), page)
                got = s["cache"][0][p, row].double() * s["cache"][2][p].double()[:, None]
                want = k[at + j].double()
                assert ((got - want).abs() <= 2.0 ** -4 * want.abs() + 2.0 ** -17 * k.double().abs().max()).all()
            at += new[i]
            if not plain[i][0] or not new[i]:
                continue
            ks, vs = (torch.stack(t) for t in plain[i])
            for h in range(Hq):
                qh = q[at - 1, h].double().cpu()
                score = ks[:, h // 4] @ qh / math.sqrt(D)
                # |e^d - 1| <= 2 d up to d = 1: the scores' error is 2^-3 sum |q||k| / sqrt(D) at most
                wide = 2.0 ** -3 * float((ks[:, h // 4].abs() @ qh.abs()).max()) / math.sqrt(D)
                p = torch.softmax(score, 0)
                off = (o[i, h].double().cpu() - p @ vs[:, h // 4]).abs()
                assert (off <= (2.0 ** -2 + 2 * wide) * (p @ vs[:, h // 4].abs()) + 1e-3).all()
                assert abs(float(l[i, h]) - float(torch.logsumexp(score, 0))) <= wide + 1e-4


def test_side_stream_and_graph():
    """All of them on a stream of their own, and captured into a graph that serves on."""
    Hq, Hkv, D, B = 8, 2, 128, 4
    r = make(9)
    prompt, steps = r(200, (Hq + 2 * Hkv) * D), [r(B, (Hq + 2 * Hkv) * D) for _ in range(5)]

    def run(graphed):
        s = serve_state(B, Hq, Hkv, D, 16, 20, 1)
        dq = torch.randn(B, Hq, D, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
        outs = [serve(s, prompt, i32([100, 60, 0, 40]), Hq, Hkv)[:2]]
        x, one = steps[0].clone(), i32([1] * B)

        def step():
            o, l, q, k, slots = serve(s, x, one, Hq, Hkv)
            raw = x[:, :Hq * D].unflatten(1, (Hq, D))
            return o, l, slots, *K.qk_norm_rope_backward(raw, None, dq, None, s["w"][0], None, s["freq"],
                                                         s["lens"])[::2]
        outs.append(step())
        graph = torch.cuda.CUDAGraph() if graphed else None
        for i in range(1, 5):
            x.copy_(steps[i])
            if graph is None:
                outs.append(step())
            else:
                if i == 1:
                    torch.cuda.current_stream().synchronize()
                    with torch.cuda.graph(graph, stream=torch.cuda.current_stream()):
                        held = step()
                if i == 3:   # a larger call on this stream takes a larger workspace
                    big = cache_case([5000] * 40, 64, 4, 128, 64)
                    K.paged_decode_fp8(*big)
                    K.page_plan(torch.zeros(60000, 1, dtype=I32, device="cuda"), *[i32([0] * 60000)] * 2, i32([]),
                                i32([0]), 16, 5)
                graph.replay()
                outs.append([t.clone() for t in held])
        torch.cuda.current_stream().synchronize()
        K.check_device_error()
        return outs

    ref = run(False)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run(True)
    for n, (a, b) in enumerate(zip(ref, got)):
        for t, u in zip(a, b):
            assert torch.equal(t, u), n


def test_two_threads_on_streams_of_their_own():
    Hq, Hkv, D, B = 8, 2, 128, 3
    r = make(11)
    xs = [r(700, (Hq + 2 * Hkv) * D) for _ in range(2)]
    new = [[500, 150, 50], [1, 300, 399]]

    def go(i):
        s = serve_state(B, Hq, Hkv, D, 16, 40, 1)
        o, l, q, k, slots = serve(s, xs[i], i32(new[i]), Hq, Hkv)
        q0 = xs[i][:, :Hq * D].unflatten(1, (Hq, D))
        dq, _, dw, _ = K.qk_norm_rope_backward(q0, None, q, None, s["w"][0], None, s["freq"],
                                               torch.arange(700, dtype=I32, device="cuda"))
        return [o, l, q, k, slots, dq, dw]

    ref = [go(i) for i in (0, 1)]
    K.check_device_error()
    failed, start = [], threading.Barrier(2)

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                start.wait()
                for _ in range(20):
                    got = go(i)
                torch.cuda.current_stream().synchronize()
                if not all(torch.equal(a, b) for a, b in zip(ref[i], got)):
                    failed.append(i)
        except Exception as e:
            failed.append(e)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    K.check_device_error()
    assert not failed
