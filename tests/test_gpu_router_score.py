"""The scored router against a 64-bit form: expert ids and grouping tables
exactly, weights within the fp32 roundings of their formula."""
import math

import pytest
import torch

import fp8_block_scaled_route_b200 as moe

pytestmark = pytest.mark.gpu

LOWEST = {torch.float32: torch.finfo(torch.float32).min, torch.bfloat16: torch.finfo(torch.bfloat16).min}


def reference(logits, k, bias, scoring, n_group, topk_group, group_top, renorm, scale):
    """(ids, weights) in 64 bits on the CPU, by the definition."""
    low, fmax = LOWEST[logits.dtype], torch.finfo(torch.float32).max
    x = logits.cpu().double()
    T, E = x.shape
    b = torch.zeros(E, dtype=torch.float64) if bias is None else bias.cpu().double()
    off = ~(x > low) | ~(b > -fmax)[None]
    x, b = x.clamp(max=fmax), b.clamp(max=fmax)
    if scoring == "sigmoid":
        p = 1.0 / (1.0 + torch.exp(-x))
    else:
        xm = x.masked_fill(off, -math.inf)
        z = torch.exp(xm - xm.max(1, keepdim=True).values)
        p = z / z.sum(1, keepdim=True)
    by = x if bias is None else p + b
    gv = by if bias is not None or group_top == 1 else p
    by, gv = (v.masked_fill(off, -math.inf) for v in (by, gv))
    gs = E // n_group
    inside = torch.ones(T, E, dtype=torch.bool)
    if n_group > 1:
        g = gv.view(T, n_group, gs).sort(dim=2, descending=True).values[:, :, :group_top]
        tot = torch.where(g == -math.inf, 0.0, g).sum(2)
        tot = torch.where(g[:, :, 0] == -math.inf, -math.inf, tot)
        best = torch.sort(tot, dim=1, descending=True, stable=True).indices[:, :topk_group]
        keep = torch.zeros(T, n_group, dtype=torch.bool).scatter_(1, best, True)
        inside = keep.repeat_interleave(gs, 1)
    ids = torch.empty(T, k, dtype=torch.int32)
    for t in range(T):
        cand = torch.nonzero(inside[t]).flatten()
        order = torch.sort(by[t, cand], descending=True, stable=True).indices[:k]
        ids[t] = cand[order].int()
    at = ids.long()
    dead = off.gather(1, at)
    xs = x.gather(1, at)
    if renorm:
        # in logarithms, so that no row of small scores loses its ratios
        lg = (-torch.nn.functional.softplus(-xs) if scoring == "sigmoid" else xs).masked_fill(dead, -math.inf)
        m = lg.max(1, keepdim=True).values
        u = torch.exp(lg - torch.where(m == -math.inf, 0.0, m))
        s = u.sum(1, keepdim=True)
        w = torch.where(s > 0, u / s, 0.0)
    else:
        w = p.gather(1, at).masked_fill(dead, 0.0)
    return ids, w * scale


def buffers(T, E, k):
    i32 = dict(dtype=torch.int32, device="cuda")
    return (torch.full((T, k), -7, **i32), torch.full((T, k), -7.0, device="cuda"),
            torch.full((E + 1,), -7, **i32), torch.full((T * k,), -7, **i32),
            torch.full((T * k,), -7, **i32),
            torch.empty(moe.moe_route_workspace_size(T, k, E), dtype=torch.uint8, device="cuda"))


def check(logits, k, bias=None, scoring="softmax", n_group=1, topk_group=1, group_top=1, renorm=True,
          scale=1.0, span=30.0):
    """Both entry points against the reference.  span: largest distance of a
    chosen logit from the largest chosen one (the exponential's argument)."""
    T, E = logits.shape
    how = dict(bias=bias, scoring=scoring, n_group=n_group, topk_group=topk_group,
               group_top=group_top, renorm=renorm, scale=scale)
    ids_r, w_r = reference(logits, k, **how)
    # renormalised: the argument's rounding (span ulps), two exponentials, a sum
    # of 32, three more operations; plain softmax: hardware exponentials (2 +
    # 1.17 * 2 ulps where they count), a 37-term sum, three operations
    rel = (span + 2 * 4 + 6 + 6) * 2.0 ** -24 if renorm or scoring == "sigmoid" else (span + 64) * 2.0 ** -24
    ids, w, m, perm, inv, ws = buffers(T, E, k)
    moe.moe_router_score_topk(logits, ids, w, **how)
    ids2, w2 = ids.clone(), w.clone()
    ids.fill_(-7)
    moe.moe_router_score_route(logits, ids, w, m, perm, inv, ws, **how)
    assert moe.moe_get_device_status(ws) == moe.MOE_OK
    assert torch.equal(ids2, ids) and torch.equal(w2, w)
    assert torch.equal(ids.cpu(), ids_r)
    d = (w.cpu().double() - w_r).abs()
    assert bool((d <= rel * w_r + 1e-37).all()), float((d / w_r.clamp(min=1e-30)).max())
    flat = ids_r.flatten().long()
    p_r = torch.sort(flat, stable=True).indices
    counts = torch.bincount(flat, minlength=E)
    assert torch.equal(m.cpu().long(), torch.cat([torch.zeros(1, dtype=torch.long), counts.cumsum(0)]))
    assert torch.equal(perm.cpu().long(), p_r)
    assert torch.equal(inv.cpu().long()[p_r], torch.arange(T * k))


SHAPES = [  # T, E, k, n_group, topk_group, group_top
    (1, 1, 1, 1, 1, 1), (1, 256, 8, 8, 4, 2), (2, 5, 5, 1, 1, 1), (33, 60, 6, 5, 2, 1),
    (64, 256, 8, 8, 4, 2), (129, 128, 8, 1, 1, 1), (200, 160, 6, 8, 3, 1), (130, 1024, 32, 32, 32, 2),
    (37, 1000, 9, 4, 1, 2), (300, 512, 16, 16, 5, 2), (1030, 64, 8, 4, 2, 2), (40, 32, 3, 32, 4, 2),
    (50, 257, 4, 1, 1, 1), (700, 300, 8, 1, 1, 1), (1100, 372, 6, 4, 3, 2), (257, 700, 31, 7, 6, 1),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,G,tg,top", SHAPES)
def test_shapes(T, E, k, G, tg, top, scoring, dtype):
    g = torch.Generator().manual_seed(T * 7 + E)
    logits = (torch.randn(T, E, generator=g) * 1.5).to(dtype).cuda()
    bias = (torch.randn(E, generator=g) * 0.1).cuda()
    for b in (None, bias):
        for renorm, scale in ((True, 2.5), (False, 1.0)):
            check(logits, k, b, scoring, G, tg, top, renorm, scale)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("G,tg,top", [(1, 1, 1), (8, 3, 1), (8, 3, 2)])
def test_ties(G, tg, top, scoring, dtype):
    """Few distinct logits and biases: equal values everywhere, by the lowest index."""
    g = torch.Generator().manual_seed(3)
    logits = (torch.randint(-2, 3, (70, 128), generator=g) * 0.5).to(dtype)
    logits[0] = 0.25
    logits[1] = -0.0
    logits[1, ::2] = 0.0
    bias = torch.randint(0, 2, (128,), generator=g) * 0.125
    for b in (None, torch.zeros(128).cuda(), bias.cuda()):
        check(logits.cuda(), 8, b, scoring, G, tg, top)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("G,tg,top", [(1, 1, 1), (4, 2, 2)])
def test_near_ties(G, tg, top, scoring):
    """Selection values that differ by less than an fp32 step of the score: the
    64-bit order decides."""
    g = torch.Generator().manual_seed(4)
    row = torch.randn(64, generator=g)
    logits = row.repeat(9, 1)
    logits[1:] += torch.randn(8, 64, generator=g) * 1e-7
    p = torch.sigmoid(row.double()) if scoring == "sigmoid" else torch.softmax(row.double(), 0)
    bias = (0.7 - p).float()
    check(logits.cuda(), 8, bias.cuda(), scoring, G, tg, top)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("G,tg,top", [(1, 1, 1), (4, 2, 1), (4, 2, 2)])
def test_masks(G, tg, top, scoring, dtype):
    g = torch.Generator().manual_seed(5)
    logits = torch.randn(12, 32, generator=g).to(dtype)
    low = LOWEST[dtype]
    logits[0] = -math.inf                     # nothing left
    logits[1] = math.nan
    logits[2] = low
    logits[3, :30] = -math.inf                # fewer experts than k
    logits[4, 3:] = low
    logits[5, ::3] = math.nan
    logits[6, 8:] = -math.inf                 # whole groups
    logits[7, 1:8] = -math.inf                # a group with one expert
    logits[8, 5] = math.inf
    logits[9, 4] = logits[9, 20] = math.inf
    bias = torch.randn(32, generator=g) * 0.1
    bias[11], bias[12], bias[13] = -math.inf, math.nan, torch.finfo(torch.float32).min
    forced = torch.zeros(32)
    forced[17] = math.inf
    for b in (None, bias, forced):
        for renorm in (True, False):
            check(logits.cuda(), 4, None if b is None else b.cuda(), scoring, G, tg, top, renorm)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_far_logits(scoring):
    """Scores that leave fp32's range keep their ratios when renormalised."""
    logits = torch.tensor([[-200.0, -201.0, -203.5, -400.0], [300.0, 299.0, 100.0, 0.0],
                           [-90.0, -95.0, -100.0, 60.0], [0.0, 1e30, -1e30, 5.0]])
    check(logits.cuda(), 3, None, scoring, span=210.0)
    check(logits.cuda(), 2, torch.tensor([0.5, 0.4, 0.3, -1.0]).cuda(), scoring, span=210.0)


@pytest.mark.parametrize("T,E,k", [(5000, 40, 1), (9000, 16, 1), (20000, 64, 8), (2049, 512, 32), (16384, 1024, 8)])
def test_many_tokens(T, E, k):
    """Each way of grouping: ids counted by the placing launch, before it, and summed up before it."""
    g = torch.Generator(device="cuda").manual_seed(T)
    logits = torch.randn(T, E, generator=g, device="cuda")
    ids, w, m, perm, inv, ws = buffers(T, E, k)
    moe.moe_router_score_route(logits, ids, w, m, perm, inv, ws)
    assert moe.moe_get_device_status(ws) == moe.MOE_OK
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    assert torch.equal(ids.long(), order.indices[:, :k])
    want = torch.softmax(order.values[:, :k].double(), 1)
    # an exponential's argument rounding (9 ulps), itself, a sum of 32, two products
    assert bool(((w.double() - want).abs() <= 48 * 2.0 ** -24 * want).all())
    flat = ids.flatten().long()
    assert torch.equal(perm.long(), torch.sort(flat, stable=True).indices)
    assert torch.equal(inv.long()[perm.long()], torch.arange(T * k, device="cuda"))
    assert torch.equal(m[1:].long(), torch.bincount(flat, minlength=E).cumsum(0)) and int(m[0]) == 0


@pytest.mark.parametrize("T,E,k", [
    (128, 1024, 32), (129, 8, 1), (129, 1024, 32),            # the last call of one launch, the first of two
    (2048, 40, 8), (2049, 40, 8), (16385, 3, 1),              # 16 and 17 chunks of 1024 pairs
    (16384, 256, 8), (16400, 256, 8), (32768, 1024, 1),       # 32768 counts of chunks, and more
    (70000, 8, 2), (262145, 64, 2), (300000, 33, 1), (40001, 500, 10)])
def test_grouping_at_its_boundaries(T, E, k):
    """Each way of grouping at its first and last sizes, a status and rows of
    counts left by an earlier call in the workspace, half of the pairs on one
    expert."""
    g = torch.Generator(device="cuda").manual_seed(T + E)
    logits = torch.randn(T, E, generator=g, device="cuda", dtype=torch.bfloat16)
    logits[::2, E // 2] = 9.0
    ids, w, m, perm, inv, ws = buffers(T, E, k)
    ws.fill_(255)
    for _ in range(2):
        perm.fill_(-7)
        inv.fill_(-7)
        moe.moe_router_score_route(logits, ids, w, m, perm, inv, ws, renorm=False)
        assert moe.moe_get_device_status(ws) == moe.MOE_OK
        flat = ids.flatten().long()
        assert torch.equal(perm.long(), torch.sort(flat, stable=True).indices)
        assert torch.equal(inv.long()[perm.long()], torch.arange(T * k, device="cuda"))
        assert torch.equal(m[1:].long(), torch.bincount(flat, minlength=E).cumsum(0)) and int(m[0]) == 0
    two, w2 = torch.full_like(ids, -7), torch.full_like(w, -7.0)
    moe.moe_router_score_topk(logits, two, w2, renorm=False)
    assert torch.equal(two, ids) and torch.equal(w2, w)
    assert bool((ids[::2, 0] == E // 2).all())


def test_no_tokens():
    ids, w, m, perm, inv, ws = buffers(0, 16, 4)
    logits = torch.empty(0, 16, device="cuda")
    assert moe.moe_router_score_topk(logits, ids, w) == moe.MOE_OK
    assert moe.moe_router_score_route(logits, ids, w, m, perm, inv, ws) == moe.MOE_OK
    assert int(m.abs().sum()) == 0 and moe.moe_get_device_status(ws) == moe.MOE_OK


def test_stream_capture_and_no_inverse():
    """On a side stream, captured, replayed on new logits, without inv_perm."""
    g = torch.Generator().manual_seed(6)
    for T in (16, 700):
        logits = torch.randn(T, 64, generator=g).cuda()
        ids, w, m, perm, _, ws = buffers(T, 64, 4)
        run = lambda: moe.moe_router_score_route(logits, ids, w, m, perm, None, ws)  # noqa: E731
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        logits.copy_(torch.randn(T, 64, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        r_ids, _ = reference(logits, 4, None, "softmax", 1, 1, 1, True, 1.0)
        assert torch.equal(ids.cpu(), r_ids)
        assert torch.equal(perm.cpu().long(), torch.sort(r_ids.flatten().long(), stable=True).indices)


@pytest.mark.parametrize("T", [5, 300])
def test_bf16_logits_at_any_element(T):
    """bf16 logits that start on an odd element, as rows cut out of a larger tensor do."""
    g = torch.Generator().manual_seed(10)
    rows = torch.randn(T + 1, 33, generator=g).bfloat16().cuda()
    assert rows[1:].data_ptr() % 4 == 2
    check(rows[1:], 4, None, "softmax")


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_group_sums_that_cancel(scoring):
    """A group's two largest values nearly cancel: their fp32 sum is rounded at
    the size of its terms, far above its own, and the chosen groups are still
    those of the 64-bit sums."""
    if scoring == "sigmoid":
        check(torch.tensor([[0.0012, 0.0012, 0.0020, 0.0]]).cuda(), 2,
              torch.tensor([1e4, -1e4, 1e4, -1e4]).cuda(), scoring, 2, 1, 2)
    g = torch.Generator().manual_seed(8)
    for big in (100.0, 1e4, 1e6):
        logits = torch.randn(600, 32, generator=g) * (1e-7 * big)
        bias = torch.tensor([big, -big]).repeat(16)
        check(logits.cuda(), 4, bias.cuda(), scoring, 16, 5, 2, span=1.0)
        # some groups cancel, some have two experts in reach, some one of them
        bias[8:16] = 0.1 * torch.randn(8, generator=g)
        bias[17:21:2] = -1e9
        check(logits.cuda(), 4, bias.cuda(), scoring, 16, 5, 2, span=1.0)
        check(logits.cuda(), 8, bias.cuda(), scoring, 8, 3, 2, span=1.0)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_group_sums_beyond_fp32(scoring):
    """Biases near fp32's ends: a group whose sum leaves fp32's range is not one
    of masked experts, and keeps its place among its like."""
    g = torch.Generator().manual_seed(9)
    logits = torch.randn(20, 15, generator=g).cuda()
    low, b16 = -3.402823466e38, float(torch.finfo(torch.bfloat16).min)
    for groups in ([low, -3e38, -2.9e38, -3.2e38, -3.1e38], [-3e38, low, low, b16, -2e38],
                   [low, b16, b16, low, b16], [3e38, 3.1e38, low, 3.2e38, -3e38], [low, -3e38, 0.5, -2e38, 3e38]):
        bias = torch.tensor(groups).repeat_interleave(3).cuda()
        for tg in (1, 2, 3, 4):
            check(logits, 3, bias, scoring, 5, tg, 2)
