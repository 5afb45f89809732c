"""The operators together, as a W8A8 expert block uses them: residual addition
and norm, scored routing, int8 rows grouped by expert, gate/up product, int8
intermediate, down product, weighted combine."""
import pytest
import torch

import fp8_block_scaled_route_b200 as moe

pytestmark = pytest.mark.gpu


def _weights(E, N, K, g):
    w = torch.randn(E, N, K, generator=g, device="cuda") / K ** 0.5
    s = w.abs().amax(2) / 127.0
    return (w / s[:, :, None]).round().to(torch.int8), s


def _rows(x):
    """int8 rows by the quantiser's formula, in 64 bits: what they stand for."""
    s = x.abs().amax(1, keepdim=True) / 127.0
    return torch.round(x / s) * s


@pytest.mark.parametrize("T,H,I,E,k", [(1, 256, 128, 8, 2), (64, 512, 256, 16, 4), (333, 512, 384, 8, 2),
                                       (1500, 256, 256, 4, 2)])
def test_block(T, H, I, E, k):
    g = torch.Generator(device="cuda").manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, res, gamma = r(T, H).bfloat16(), r(T, H).bfloat16(), 1 + 0.1 * r(H)
    gate_w, bias = r(E, H) / H ** 0.5, 0.1 * r(E)
    (w13, s13), (w2, s2) = _weights(E, 2 * I, H, g), _weights(E, H, I, g)
    R = T * k
    i32 = dict(dtype=torch.int32, device="cuda")
    y, h = torch.empty_like(x), torch.empty_like(x)
    ids, w = torch.empty(T, k, **i32), torch.empty(T, k, device="cuda")
    m, perm, inv = torch.empty(E + 1, **i32), torch.empty(R, **i32), torch.empty(R, **i32)
    ws = torch.empty(moe.moe_route_workspace_size(T, k, E), dtype=torch.uint8, device="cuda")
    xq, xs = torch.empty(R, H, dtype=torch.int8, device="cuda"), torch.empty(R, device="cuda")
    hid = torch.empty(R, I, dtype=torch.bfloat16, device="cuda")
    hq, hs = torch.empty(R, I, dtype=torch.int8, device="cuda"), torch.empty(R, device="cuda")
    rows, out = torch.empty(R, H, device="cuda"), torch.empty_like(x)
    logits = torch.empty(T, E, device="cuda")

    def run():
        moe.moe_rmsnorm_quant(x, gamma, 1e-6, residual=res, residual_out=h, y=y)
        torch.matmul(y.float(), gate_w.t(), out=logits)
        moe.moe_router_score_route(logits, ids, w, m, perm, inv, ws, bias=bias, scoring="sigmoid",
                                   n_group=2, topk_group=2, group_top=2, scale=1.5)
        moe.int8_quantize(y, xq, xs, inv_perm=inv, k=k)
        moe.int8_moe_gemm(xq, w13, xs, s13, hid, m_indptr=m, is_gated=True)
        moe.int8_quantize(hid, hq, hs)
        moe.int8_moe_gemm(hq, w2, hs, s2, rows, m_indptr=m)
        moe.moe_combine(rows, inv, w, out)

    run()
    assert moe.moe_get_device_status(ws) == moe.MOE_OK and moe.moe_get_device_status(None) == moe.MOE_OK
    first = out.clone()
    # the same block in 64 bits from the operators' own y, ids and weights (each
    # of which has its own test)
    d = h.double()
    y64 = d / torch.sqrt(d.square().mean(1, keepdim=True) + 1e-6) * gamma.double()
    assert float((y.double() - y64).norm() / y64.norm()) < 2.0 ** -8
    want = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    xr = _rows(y.double())
    for j in range(k):
        for e in range(E):
            t = torch.nonzero(ids[:, j] == e).flatten()
            if t.numel() == 0:
                continue
            v = xr[t] @ (w13[e].double() * s13[e].double()[:, None]).t()
            mid = v[:, :I] * torch.sigmoid(v[:, :I]) * v[:, I:]
            mid = _rows(mid.bfloat16().double())
            want[t] += w[t, j, None].double() * (mid @ (w2[e].double() * s2[e].double()[:, None]).t())
    # differences: the output's bf16 rounding (2^-8 at most, about 2^-9.8 in the
    # norm) and int8 codes of the intermediate that a bf16 rounding moves by a
    # step (1/127 of the row's largest value, on a few values of a row)
    assert float((out.double() - want).norm() / want.norm()) < 2.0 ** -8
    # captured and replayed, the block gives the same bits
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        run()
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)


def _layers(T, H, I, E, k, seed):
    """Eight chained blocks on one set of buffers, the residual stream updated in
    place; run(x, each) calls each() after every operator."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    (w13, s13), (w2, s2) = _weights(E, 2 * I, H, g), _weights(E, H, I, g)
    gamma, bias, gate_w, R = 1 + 0.1 * r(H), 0.1 * r(E), r(E, H) / H ** 0.5, T * k
    i32 = dict(dtype=torch.int32, device="cuda")
    h, y, out = (torch.zeros(T, H, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    ids, w = torch.empty(T, k, **i32), torch.empty(T, k, device="cuda")
    m, perm, inv = torch.empty(E + 1, **i32), torch.empty(R, **i32), torch.empty(R, **i32)
    ws = torch.empty(moe.moe_route_workspace_size(T, k, E), dtype=torch.uint8, device="cuda")
    xq, xs = torch.empty(R, H, dtype=torch.int8, device="cuda"), torch.empty(R, device="cuda")
    hid = torch.empty(R, I, dtype=torch.bfloat16, device="cuda")
    hq, hs = torch.empty(R, I, dtype=torch.int8, device="cuda"), torch.empty(R, device="cuda")
    rows, logits = torch.empty(R, H, device="cuda"), torch.empty(T, E, device="cuda")
    calls = [
        lambda: moe.moe_rmsnorm_quant(out, gamma, 1e-6, residual=h, residual_out=h, y=y),
        lambda: torch.matmul(y.float(), gate_w.t(), out=logits),
        lambda: moe.moe_router_score_route(logits, ids, w, m, perm, inv, ws, bias=bias, scoring="sigmoid",
                                           n_group=2, topk_group=1, group_top=2),
        lambda: moe.int8_quantize(y, xq, xs, inv_perm=inv, k=k),
        lambda: moe.int8_moe_gemm(xq, w13, xs, s13, hid, m_indptr=m, is_gated=True),
        lambda: moe.int8_quantize(hid, hq, hs),
        lambda: moe.int8_moe_gemm(hq, w2, hs, s2, rows, m_indptr=m),
        lambda: moe.moe_combine(rows, inv, w, out)]

    def run(x, each=lambda: None):
        h.copy_(x)
        out.copy_(x)
        for _ in range(8):
            for call in calls:
                call()
                each()
        return h.clone(), out.clone(), perm.clone()
    return run


@pytest.mark.parametrize("T,H,I,E,k", [(4, 512, 256, 16, 4), (64, 256, 256, 32, 8), (200, 512, 256, 8, 2),
                                       (3000, 256, 256, 64, 6)])
def test_chained_blocks_on_two_streams(T, H, I, E, k):
    """Each operator may start before its predecessor has ended: chained calls
    without a pause, on two streams at once, give the bits of calls that wait."""
    a, b = _layers(T, H, I, E, k, 1), _layers(T, H, I, E, k, 2)
    g = torch.Generator(device="cuda").manual_seed(T)
    xs = [torch.randn(T, H, generator=g, device="cuda").bfloat16() for _ in range(3)]
    want = [run(x, torch.cuda.synchronize) for x in xs for run in (a, b)]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        torch.cuda.synchronize()
        got = []
        for x in xs:
            for run, stream in ((a, s1), (b, s2)):
                with torch.cuda.stream(stream):
                    got.append(run(x))
        torch.cuda.synchronize()
        for u, v in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(u, v))
    assert moe.moe_get_device_status(None) == moe.MOE_OK


def test_norm_rows_feed_the_block_scaled_gemms():
    """The norm's FP8 and MXFP8 rows, in both scale layouts, as the activation
    operand of the existing grouped GEMMs."""
    T, H, N = 200, 512, 256
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    gamma = torch.ones(H, device="cuda")
    wq = torch.randn(1, N, H, generator=g, device="cuda").to(torch.float8_e4m3fn)
    m = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    d = x.double()
    y64 = d / torch.sqrt(d.square().mean(1, keepdim=True) + 1e-6)
    want = y64 @ wq[0].double().t()
    u8 = dict(dtype=torch.uint8, device="cuda")
    tiled = torch.empty(N * H // 32, **u8)
    moe.mxfp8_tile_scales(torch.full((N, H // 32), 127, **u8), tiled)
    for mn in (False, True):
        major = "MN" if mn else "K"
        q = torch.empty(T, H, dtype=torch.float8_e4m3fn, device="cuda")
        s = torch.empty((H // 128, T) if mn else (T, H // 128), device="cuda")
        sf = torch.empty((H // 128, T, 4) if mn else (T, H // 32), **u8)
        out = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
        moe.moe_rmsnorm_quant(x, gamma, 1e-6, q_format="fp8", q=q, q_scale=s, scale_major=major)
        moe.fp8_groupwise_moe_gemm(q, wq, s, torch.ones(1, N // 128, H // 128, device="cuda"), m, out,
                                   scale_major_mode=major)
        # E4M3 values are off by 2^-4 at most, so products of independent ones by
        # less than that in the norm
        assert float((out.double() - want).norm() / want.norm()) < 2.0 ** -4
        moe.moe_rmsnorm_quant(x, gamma, 1e-6, q_format="mxfp8", q=q, q_scale=sf, scale_major=major)
        moe.mxfp8_moe_gemm(q, wq, sf, tiled, m, out, a_sf_major=major)
        assert float((out.double() - want).norm() / want.norm()) < 2.0 ** -4


def test_inputs_rewritten_by_the_kernel_before():
    """Each operator may be resident before its predecessor has ended, and reads
    what that one writes: norm weights, rows and destination rows rewritten by
    the call before, without a pause, give the bits of calls that wait."""
    T, H, E, k, n = 64, 1024, 16, 2, 48
    g = torch.Generator(device="cuda").manual_seed(12)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    gammas, xs, logits = r(6, 1, H).bfloat16(), r(6, T, H).bfloat16(), r(6, T, E)
    ones, i32 = torch.ones(H, device="cuda"), dict(dtype=torch.int32, device="cuda")
    weight = torch.zeros(1, H, dtype=torch.bfloat16, device="cuda")
    y = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    ids, w, m = torch.empty(T, k, **i32), torch.empty(T, k, device="cuda"), torch.empty(E + 1, **i32)
    perm, inv = torch.zeros(T * k, **i32), torch.zeros(T * k, **i32)
    ws = torch.empty(moe.moe_route_workspace_size(T, k, E), dtype=torch.uint8, device="cuda")

    def run(each=lambda: None):
        q = torch.zeros(n, T * k, H, dtype=torch.int8, device="cuda")
        s, ys = torch.zeros(n, T * k, device="cuda"), torch.zeros(n, T, H, dtype=torch.bfloat16, device="cuda")
        q1, s1 = torch.zeros(n, T, H, dtype=torch.int8, device="cuda"), torch.zeros(n, T, device="cuda")
        for i in range(n):
            j = i % 6
            for call in (lambda: moe.moe_rmsnorm_quant(gammas[j], ones, 1e-6, y=weight),
                         lambda: moe.moe_rmsnorm_quant(xs[j], weight[0], 1e-6, y=ys[i]),
                         lambda: moe.moe_rmsnorm_quant(xs[-j], weight[0], 1e-6, y=y),
                         lambda: moe.int8_quantize(y, q1[i], s1[i]),
                         lambda: moe.moe_router_score_route(logits[j], ids, w, m, perm, inv, ws),
                         lambda: moe.int8_quantize(y, q[i], s[i], inv_perm=inv, k=k)):
                call()
                each()
        torch.cuda.synchronize()
        return q, s, ys, q1, s1

    want = run(torch.cuda.synchronize)
    for _ in range(4):
        assert all(torch.equal(a, b) for a, b in zip(run(), want))


def test_first_call_of_a_thread():
    """Each operator as a new thread's first use of the GPU: a thread that no call
    of the CUDA runtime has bound to a context yet."""
    import threading
    T, H, E, k = 8, 256, 4, 2
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, gamma, logits = r(T, H).bfloat16(), torch.ones(H, device="cuda"), r(T, E)
    y, out = torch.empty_like(x), torch.empty(T, 64, dtype=torch.bfloat16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    ids, w, m = torch.empty(T, k, **i32), torch.empty(T, k, device="cuda"), torch.empty(E + 1, **i32)
    perm, ws = torch.empty(T * k, **i32), torch.empty(moe.moe_route_workspace_size(T, k, E), dtype=torch.uint8,
                                                      device="cuda")
    q, s = torch.empty(T, H, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    (b, sb), stream = _weights(1, 64, H, g), torch.cuda.Stream()
    moe.int8_quantize(x, q, s)
    torch.cuda.synchronize()
    calls = [lambda h: moe.moe_rmsnorm_quant(x, gamma, 1e-6, y=y, stream=h),
             lambda h: moe.moe_router_score_topk(logits, ids, w, stream=h),
             lambda h: moe.moe_router_score_route(logits, ids, w, m, perm, None, ws, stream=h),
             lambda h: moe.int8_quantize(x, q, s, stream=h),
             lambda h: moe.int8_moe_gemm(q, b, s, sb, out, stream=h)]
    for i, call in enumerate(calls):
        got = []

        def run(call=call):
            try:
                got.append(call(stream.cuda_stream))
            except Exception as e:  # noqa: BLE001  (told to the test's own thread)
                got.append(e)

        t = threading.Thread(target=run)
        t.start()
        t.join()
        torch.cuda.synchronize()
        assert got == [moe.MOE_OK], (i, got)
