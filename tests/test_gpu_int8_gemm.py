"""The grouped int8 GEMM against exact integer sums (64-bit products on the
GPU), with the roundings of its epilogue counted."""
import pytest
import torch

import fp8_block_scaled_route_b200 as moe

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def make(R, N, K, E, seed, extreme=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    lo = -128
    a = torch.randint(lo, 128, (R, K), generator=g, device="cuda", dtype=torch.int8)
    b = torch.randint(lo, 128, (E, N, K), generator=g, device="cuda", dtype=torch.int8)
    if extreme:
        a.fill_(-128)
        b[:, ::2] = -128
        b[:, 1::2] = 127
    sa = 0.01 + torch.rand(R, generator=g, device="cuda")
    sb = (0.5 + torch.rand(E, N, generator=g, device="cuda")) / (5000.0 * K ** 0.5)
    return a, b, sa, sb


def reference(a, b, sa, sb, edges, gated):
    """(out in 64 bits, tolerance without the output's own rounding)"""
    R, N = a.shape[0], b.shape[1]
    n = N // 2 if gated else N
    out = torch.zeros(R, n, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(out)
    for e in range(b.shape[0]):
        lo, hi = edges[e], edges[e + 1]
        if hi <= lo:
            continue
        s = a[lo:hi].double() @ b[e].double().t()      # exact: below 2^53
        v = s * sa[lo:hi, None].double() * sb[e].double()
        if not gated:
            out[lo:hi] = v
            tol[lo:hi] = 4 * U * v.abs()               # the sum to fp32 and two products
        else:
            g, u = v[:, :n], v[:, n:]
            out[lo:hi] = g * torch.sigmoid(g) * u
            # g off by 3 U: silu by 3 |g| U and 3 U, the hardware exponential by (2 +
            # 1.17 |g|) ulps, its sum, reciprocal, and two products; u by 3 U
            tol[lo:hi] = (6 * g.abs() + 24) * U * out[lo:hi].abs() + 1e-35 * (1 + u.abs())
    return out, tol


def check(R, N, K, E, gated=False, dtype=torch.bfloat16, counts=None, seed=0, extreme=False, dense=False):
    a, b, sa, sb = make(R, N, K, E, seed, extreme)
    if counts is None:
        g = torch.Generator().manual_seed(seed + 1)
        counts = torch.bincount(torch.randint(0, E, (R,), generator=g), minlength=E).tolist()
    edges = [0]
    for c in counts:
        edges.append(edges[-1] + c)
    assert edges[-1] <= R
    n = N // 2 if gated else N
    out = torch.full((R + 2, n), -77.0, dtype=dtype, device="cuda")
    m = None if dense else torch.tensor(edges, dtype=torch.int32, device="cuda")
    moe.int8_moe_gemm(a, b, sa, sb, out[:R], m_indptr=m, is_gated=gated)
    assert moe.moe_get_device_status(None) == moe.MOE_OK
    ref, tol = reference(a, b, sa, sb, edges, gated)
    used = edges[-1]
    if dtype is torch.bfloat16:
        tol = tol + ref.abs() * 2.0 ** -8 + 2.0 ** -133
    d = (out[:used].double() - ref[:used]).abs()
    bad = d > tol[:used]
    assert not bool(bad.any()), (int(bad.sum()), torch.nonzero(bad)[:4].tolist(), float(d.max()))
    assert bool((out[used:] == -77).all())             # rows behind the last expert's
    return a, b, sa, sb, out


DENSE = [  # R, N, K
    (1, 1, 16), (1, 128, 128), (1, 4096, 7168), (2, 33, 48), (15, 130, 144), (16, 64, 2048), (17, 256, 640),
    (33, 1000, 272), (64, 512, 1024), (65, 513, 128), (128, 384, 7168), (129, 258, 2000), (300, 1024, 512),
    (511, 640, 4096), (1000, 2048, 256), (2050, 1030, 1040), (4096, 512, 384),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R,N,K", DENSE)
def test_dense(R, N, K, dtype):
    check(R, N, K, 1, dtype=dtype, counts=[R], dense=True)
    if N % 2 == 0:
        check(R, N, K, 1, gated=True, dtype=dtype, counts=[R], dense=True)


GROUPED = [  # R, N, K, E
    (1, 64, 64, 8), (7, 256, 128, 4), (64, 200, 272, 16), (100, 384, 512, 128), (512, 1536, 2048, 16),
    (1000, 258, 640, 3), (3000, 512, 256, 5), (5000, 130, 144, 20), (2048, 1024, 1024, 2), (40, 128, 64, 1024),
]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("R,N,K,E", GROUPED)
def test_grouped(R, N, K, E, gated):
    check(R, N, K, E, gated)
    check(R, N, K, E, gated, dtype=torch.float32, seed=5)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("counts", [
    [0, 0, 5, 0], [700, 0, 0, 1], [0, 1, 17, 600], [256, 128, 384, 16], [1, 0, 0, 0], [0, 0, 0, 0],
    [255, 257, 1, 129], [3000, 1, 2, 900],
])
def test_skewed_and_empty(counts, gated):
    """Experts without rows, one that has nearly all, and rows behind the last."""
    check(sum(counts) + 9, 320, 336, 4, gated, counts=counts, seed=2)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("R,N,K", [(20, 256, 1024), (100, 512, 4096), (300, 512, 4096), (520, 640, 2048),
                                   (2000, 256, 256)])
def test_one_expert_with_fewer_rows(R, N, K, gated):
    """One expert whose m_indptr names some of the R rows, or none of them."""
    for n in (0, 1, R // 2, R - 1):
        check(R, N, K, 1, gated, counts=[n], seed=n)


@pytest.mark.parametrize("R", [3, 600])
def test_largest_sums(R):
    """-128 * -128 over the longest K whose 32-bit sums cannot overflow."""
    check(R, 64, 131056, 1, dtype=torch.float32, counts=[R], extreme=True, dense=True)


def test_bad_m_indptr_stays_in_bounds():
    """A table outside [0, R] or decreasing is clamped: no row past R is touched."""
    a, b, sa, sb = make(40, 64, 128, 3, 1)
    for edges in ([0, 10, 60, 60], [-5, 10, 20, 40], [0, 30, 10, 40]):
        out = torch.full((44, 64), -77.0, dtype=torch.bfloat16, device="cuda")
        moe.int8_moe_gemm(a, b, sa, sb, out[:40], m_indptr=torch.tensor(edges, dtype=torch.int32, device="cuda"))
        assert moe.moe_get_device_status(None) == moe.MOE_OK
        assert bool((out[40:] == -77).all())


def test_special_scales():
    """Infinite and NaN scales stay in their own rows and channels."""
    a, b, sa, sb = make(20, 96, 128, 1, 3)
    sa[3], sb[0, 70] = float("nan"), float("inf")
    out = torch.empty(20, 96, device="cuda")
    moe.int8_moe_gemm(a, b, sa, sb, out)
    bad = ~torch.isfinite(out)
    want = torch.zeros_like(bad)
    want[3] = True
    want[:, 70] = True
    zero = (a.double() @ b[0].double().t()) == 0
    assert torch.equal(bad, want | (zero & want))


def test_no_rows():
    a, b, sa, sb = make(4, 64, 64, 2, 1)
    out = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    m = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert moe.int8_moe_gemm(a[:0], b, sa[:0], sb, out, m_indptr=m) == moe.MOE_OK


@pytest.mark.parametrize("R,N,K,E", [(3, 512, 2048, 1), (200, 256, 512, 8), (2000, 512, 512, 2)])
def test_runs_are_identical_streams_and_capture(R, N, K, E):
    """The same bits on another stream, from two streams at once and from a graph."""
    a, b, sa, sb, out = check(R, N, K, E)
    g = torch.Generator().manual_seed(1)
    counts = torch.bincount(torch.randint(0, E, (R,), generator=g), minlength=E)
    m = torch.cat([torch.zeros(1, dtype=torch.long), counts.cumsum(0)]).int().cuda()
    outs = [torch.empty_like(out[:R]) for _ in range(3)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s, o in zip(streams, outs):
        s.wait_stream(torch.cuda.current_stream())
        moe.int8_moe_gemm(a, b, sa, sb, o, m_indptr=m, stream=s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.int8_moe_gemm(a, b, sa, sb, outs[2], m_indptr=m)
    graph.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, out[:R])


def test_wait_bound_is_reported_once():
    """A 1 ns bound on the pipeline's waits: the call ends with a status that
    stays until it is read and is gone afterwards; later calls work."""
    a, b, sa, sb = make(300, 512, 4096, 1, 3)
    out = torch.empty(300, 512, dtype=torch.bfloat16, device="cuda")
    try:
        moe.moe_set_wait_timeout_ns(1)
        moe.int8_moe_gemm(a, b, sa, sb, out)
    finally:
        moe.moe_set_wait_timeout_ns(2_000_000_000)
    assert moe.moe_get_device_status(None) == moe.MOE_ERR_DEVICE_TIMEOUT
    assert moe.moe_get_device_status(None) == moe.MOE_OK
    check(300, 512, 4096, 1, counts=[300], seed=3, dense=True)


@pytest.mark.parametrize("R,n", [(3, 64), (40, 33), (200, 64), (520, 96)])
def test_gated_fp32_output_over_the_range(R, n):
    """fp32 output of the gated product for gates from -100 to 100: SiLU within
    a few roundings of its value, however far the gate."""
    K = 16
    a = torch.zeros(R, K, dtype=torch.int8, device="cuda")
    a[:, 3] = 1
    b = torch.zeros(1, 2 * n, K, dtype=torch.int8, device="cuda")
    g = torch.Generator().manual_seed(R)
    b[0, :, 3] = torch.randint(1, 128, (2 * n,), generator=g).to(torch.int8)
    b[0, :n, 3] *= (1 - 2 * (torch.arange(n) % 2)).to(torch.int8).cuda()
    sa = (torch.rand(R, generator=g) * 0.8).cuda()
    sb = torch.ones(1, 2 * n, device="cuda")
    out = torch.empty(R, n, device="cuda")
    moe.int8_moe_gemm(a, b, sa, sb, out, is_gated=True)
    G = b[0, :, 3].float() * sa[:, None]               # the fp32 values, sums of one product
    gate, up = G[:, :n].double(), G[:, n:].double()
    want = gate * torch.sigmoid(gate) * up
    assert float(gate.min()) < -60 and float(gate.max()) > 60
    # z e / (1 + e) with e = exp(-|z|): the exponential by 4 U, its correction by 1 and
    # by ln 2's rounding (0.05 |z|), the sum by 1, the reciprocal by 2, two products
    # and that with `up`; below 2^-126 the exponential loses bits (2^-148)
    tol = (11 + 0.05 * gate.abs()) * U * want.abs() + 2.0 ** -147 * 100 * up.abs()
    d = (out.double() - want).abs()
    assert bool((d <= tol).all()), float((d / want.abs().clamp(min=1e-30)).max() / U)


def _run_out(a, b, sa, sb, out):
    """A call whose waits run out."""
    try:
        moe.moe_set_wait_timeout_ns(1)
        moe.int8_moe_gemm(a, b, sa, sb, out)
        torch.cuda.synchronize()
    finally:
        moe.moe_set_wait_timeout_ns(2_000_000_000)


def test_status_reaches_every_thread():
    """A timeout that one thread reads and clears is still told to the thread
    whose call it was, once."""
    import threading
    a, b, sa, sb = make(40, 256, 2048, 1, 4)
    out = torch.empty(40, 256, dtype=torch.bfloat16, device="cuda")
    ran, read, got = threading.Event(), threading.Event(), []

    def caller():
        torch.cuda.set_device(0)
        _run_out(a, b, sa, sb, out)
        ran.set()
        read.wait(60)
        got.extend(moe.moe_get_device_status(None) for _ in range(2))

    assert moe.moe_get_device_status(None) == moe.MOE_OK
    t = threading.Thread(target=caller)
    t.start()
    assert ran.wait(60)
    first = [moe.moe_get_device_status(None) for _ in range(2)]
    read.set()
    t.join()
    assert first == [moe.MOE_ERR_DEVICE_TIMEOUT, moe.MOE_OK]
    assert got == [moe.MOE_ERR_DEVICE_TIMEOUT, moe.MOE_OK]

    def later():     # a thread whose calls come after all that
        moe.int8_moe_gemm(a, b, sa, sb, out)
        got.append(moe.moe_get_device_status(None))

    t = threading.Thread(target=later)
    t.start()
    t.join()
    assert got[2:] == [moe.MOE_OK]


def test_status_is_not_hidden_by_the_fp8_word():
    """With both words set each is reported: the int8 one once, the other until
    its entry point's next call."""
    import synth
    inp = synth.make_grouped_gemm_inputs(0, 256, 512, 2, seed=3, group_sizes=[30, 7], device="cuda")
    fp8_out = torch.zeros(37, 128, dtype=torch.bfloat16, device="cuda")
    fp8 = lambda: moe.fp8_groupwise_moe_gemm(inp["a"], inp["b"], inp["a_scale"], inp["b_scale"],  # noqa: E731
                                             inp["m_indptr"], fp8_out, "K", (1, 128, 128), True, -1, -1)
    a, b, sa, sb = make(40, 256, 2048, 1, 4)
    out = torch.empty(40, 256, dtype=torch.bfloat16, device="cuda")
    try:
        moe.moe_set_wait_timeout_ns(1)
        fp8()
        torch.cuda.synchronize()
    finally:
        moe.moe_set_wait_timeout_ns(2_000_000_000)
    _run_out(a, b, sa, sb, out)
    assert moe.moe_get_device_status(None) == moe.MOE_ERR_DEVICE_TIMEOUT
    assert moe.moe_get_device_status(None) == moe.MOE_ERR_DEVICE_TIMEOUT
    fp8()
    assert moe.moe_get_device_status(None) == moe.MOE_OK


@pytest.mark.parametrize("R,N,K,E", [(20, 256, 4096, 1), (1000, 384, 640, 20), (4000, 1024, 512, 4)])
def test_wait_bound_on_the_other_paths(R, N, K, E):
    """A 1 ns bound on the waits of tiles split over a cluster, of the walk over an
    item table and of the persistent CTA pairs."""
    a, b, sa, sb = make(R, N, K, E, 3)
    out = torch.empty(R, N, dtype=torch.bfloat16, device="cuda")
    m = torch.arange(E + 1, dtype=torch.int32, device="cuda") * (R // E)
    try:
        moe.moe_set_wait_timeout_ns(1)
        moe.int8_moe_gemm(a, b, sa, sb, out, m_indptr=m)
    finally:
        moe.moe_set_wait_timeout_ns(2_000_000_000)
    assert moe.moe_get_device_status(None) == moe.MOE_ERR_DEVICE_TIMEOUT
    assert moe.moe_get_device_status(None) == moe.MOE_OK
    check(R, N, K, E, seed=3)
