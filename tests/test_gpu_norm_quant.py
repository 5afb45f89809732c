"""RMS norm with residual and 8-bit rows, and the int8 row quantiser, against
64-bit forms.  A rounding is off by at most half a step; each tolerance counts
the roundings of the formula."""
import math

import pytest
import torch

import fp8_block_scaled_route_b200 as moe

pytestmark = pytest.mark.gpu

U = 2.0 ** -24     # half a step of fp32, relative
TINY = 2.0 ** -100


def div(a, b):
    """a / b correctly rounded: with a Python number as an operand torch would
    multiply by a reciprocal."""
    return (a if torch.is_tensor(a) else torch.full_like(b, a)) / (b if torch.is_tensor(b) else
                                                                  torch.full_like(a, b))


def make(T, H, seed, wdtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = (r(T, H) * torch.exp(r(T, 1))).bfloat16()
    res = (3 * r(T, H)).bfloat16()
    w = (1 + 0.2 * r(H)).to(wdtype)
    return x, res, w


def reference(x, res, w, eps):
    """(h bf16, y in 64 bits)"""
    h = x if res is None else (x.float() + res.float()).bfloat16()
    d = h.double()
    return h, d / torch.sqrt(d.square().mean(1, keepdim=True) + eps) * w.double()


def check_y(y, y64):
    # r and two products in fp32, then bf16
    tol = y64.abs() * (2.0 ** -8 + 4 * U) + 2.0 ** -133
    assert bool(((y.double() - y64).abs() <= tol).all())


def check_codes(val, scale, y64, half_rel, half_abs):
    """val * scale within half a step of y64: half_rel of the value or half_abs
    scaled steps, whichever is larger, and six fp32 roundings."""
    v = val.double() * scale
    tol = torch.maximum(half_rel * y64.abs(), half_abs * scale.expand_as(y64)) * (1 + 2.0 ** -18)
    assert bool(((v - y64).abs() <= tol + 6 * U * y64.abs()).all())


def outputs(T, H, fmt, mn):
    q = torch.full((T + 2, H), 77, dtype=torch.int8 if fmt == "int8" else torch.uint8, device="cuda")
    f32 = dict(dtype=torch.float32, device="cuda")
    s = {"fp8": lambda: torch.full((H // 128, T) if mn else (T, H // 128), -5.0, **f32),
         "mxfp8": lambda: torch.full((H // 128, T, 4) if mn else (T, H // 32), 77, dtype=torch.uint8,
                                     device="cuda"),
         "int8": lambda: torch.full((T,), -5.0, **f32)}[fmt]()
    return q, s


def check_rows(fmt, mn, q, s, y64):
    """8-bit rows q and scales s of the 64-bit rows y64."""
    T, H = y64.shape
    if fmt == "int8":
        amax = y64.abs().amax(1)
        assert bool(((s.double() - amax / 127).abs() <= 5 * U * amax / 127).all())
        check_codes(q.float(), s.double()[:, None], y64, 0.0, 0.5)
        assert int(q.min()) >= -127
        return
    blk = 128 if fmt == "fp8" else 32
    amax = y64.view(T, -1, blk).abs().amax(2)
    val = q.view(torch.float8_e4m3fn).float()
    if fmt == "fp8":
        sc = (s.t() if mn else s).double()
        assert bool(((sc - amax / 448).abs() <= 5 * U * amax / 448).all())
    else:
        code = (s.transpose(0, 1).reshape(T, -1) if mn else s).int()
        sc = torch.exp2(code.double() - 127)
        live = code > 0
        assert bool((amax * (1 - 6 * U) <= 448 * sc)[live].all())         # large enough
        assert bool((amax * (1 + 6 * U) > 224 * sc)[live].all())          # and no larger
    check_codes(val, sc.repeat_interleave(blk, 1), y64, 2.0 ** -4, 2.0 ** -10)


SIZES = [(1, 128), (1, 7168), (3, 256), (17, 384), (64, 7168), (149, 2048), (300, 128), (5, 16384),
         (2, 32768), (1025, 640), (33, 4096), (7, 1152)]


@pytest.mark.parametrize("fmt", ["none", "fp8", "mxfp8", "int8"])
@pytest.mark.parametrize("T,H", SIZES)
def test_norm(T, H, fmt):
    for wdtype, use_res, mn in ((torch.float32, True, False), (torch.bfloat16, False, True)):
        x, res, w = make(T, H, T + H, wdtype)
        res = res if use_res else None
        h, y64 = reference(x, res, w, 1e-5)
        y = torch.full((T + 2, H), 9.0, dtype=torch.bfloat16, device="cuda")
        ho = torch.full((T + 2, H), 9.0, dtype=torch.bfloat16, device="cuda")
        q, s = outputs(T, H, fmt, mn) if fmt != "none" else (None, None)
        moe.moe_rmsnorm_quant(x, w, 1e-5, residual=res, residual_out=ho[:T] if use_res else None, y=y[:T],
                              q_format=fmt, q=q[:T] if q is not None else None, q_scale=s,
                              scale_major="MN" if mn else "K")
        check_y(y[:T], y64)
        if use_res:
            assert torch.equal(ho[:T], h)
        if q is not None:
            check_rows(fmt, mn, q[:T], s, y64)
            assert bool((q[T:] == 77).all())
        assert bool((y[T:] == 9).all()) and bool((ho[T:] == 9).all())     # rows behind the last one


@pytest.mark.parametrize("T,H", [(9, 16), (40, 48), (3, 2000), (260, 272), (5, 8176)])
def test_norm_int8_odd_widths(T, H):
    x, res, w = make(T, H, 1)
    _, y64 = reference(x, res, w, 1e-6)
    q, s = outputs(T, H, "int8", False)
    moe.moe_rmsnorm_quant(x, w, 1e-6, residual=res, q_format="int8", q=q[:T], q_scale=s)
    check_rows("int8", False, q[:T], s, y64)


@pytest.mark.parametrize("T,H", [(1, 7168), (200, 7168), (3, 2048), (500, 640), (4, 32768)])
def test_int8_codes_do_not_depend_on_the_split(T, H):
    """The codes are those of the elementwise fp32 formula with a 64-bit mean
    square, bit for bit, whatever number of threads shares a row."""
    x, res, w = make(T, H, 2)
    h = (x.float() + res.float()).bfloat16()
    r = div(1.0, torch.sqrt(div(h.double().square().sum(1, keepdim=True), H) + 1e-6)).float()
    y = h.float() * r * w
    amax = y.abs().amax(1)
    q, s = outputs(T, H, "int8", False)
    moe.moe_rmsnorm_quant(x, w, 1e-6, residual=res, q_format="int8", q=q[:T], q_scale=s)
    assert torch.equal(s, div(amax, 127.0))
    assert torch.equal(q[:T], torch.round(y * div(127.0, amax)[:, None]).to(torch.int8))


def test_norm_in_place():
    x, res, w = make(65, 1024, 3)
    h, y64 = reference(x, res, w, 1e-6)
    moe.moe_rmsnorm_quant(x, w, 1e-6, residual=res, residual_out=res, y=x)
    assert torch.equal(res, h)
    check_y(x, y64)


@pytest.mark.parametrize("fmt", ["fp8", "mxfp8", "int8"])
def test_norm_special_rows(fmt):
    T, H = 8, 256
    x, _, w = make(T, H, 4)
    x[0] = 0
    x[1, :128] = 0
    x[2] = 1e-38
    x[3, 5] = math.nan
    x[4, 7] = math.inf
    x[5] = 2.0 ** 100
    w[200:] = 0
    eps = 1e-6
    q, s = outputs(T, H, fmt, False)
    y = torch.empty_like(x)
    moe.moe_rmsnorm_quant(x, w, eps, y=y, q_format=fmt, q=q[:T], q_scale=s)
    fine = torch.tensor([0, 1, 5, 6, 7], device="cuda")
    # row 2: y = 1e-38 / sqrt(eps) is below 2^-100 and counts as zero
    _, y64 = reference(x, None, w, eps)
    check_y(y[fine], y64[fine])
    qf = (q[:T] if fmt == "int8" else q[:T].view(torch.float8_e4m3fn)).float()
    assert bool((qf[0] == 0).all())
    if fmt == "int8":
        assert s[0] == 1 and s[2] == 1 and bool((qf[2] == 0).all())
        assert bool(torch.isnan(s[3:5]).all()) and bool((q[3:5] == 0).all())
        check_rows(fmt, False, q[5:T], s[5:], y64[5:])
    elif fmt == "fp8":
        assert bool((s[0] == 1).all()) and bool((s[2] == 1).all()) and bool((qf[2] == 0).all())
        assert bool(torch.isnan(s[3]).all()) and bool(torch.isnan(s[4, 0]))
        check_rows(fmt, False, q[5:T], s[5:], y64[5:])
    else:
        assert bool((s[0] == 0).all()) and bool((s[3] == 255).all()) and int(s[4, 0]) == 255
        check_rows(fmt, False, q[5:T], s[5:], y64[5:])
    assert bool(torch.isnan(y[3]).all()) and bool(torch.isnan(y[4, 7]))


def test_norm_small_mean_needs_eps():
    """Rows far below eps: r is 1 / sqrt(eps), not an infinity."""
    x = torch.full((2, 128), 2.0 ** -60, dtype=torch.bfloat16, device="cuda")
    w, y = torch.ones(128, device="cuda"), torch.empty(2, 128, dtype=torch.bfloat16, device="cuda")
    moe.moe_rmsnorm_quant(x, w, 1e-12, y=y)
    check_y(y, reference(x, None, w, 1e-12)[1])


def codes64(x):
    """The quantiser's formula elementwise: (codes, scales), exact in fp32 torch."""
    f = x.float()
    amax = f.abs().amax(1)
    zero = amax < TINY
    inv = torch.where(zero, 0.0, div(127.0, amax))
    return torch.round(f * inv[:, None]).to(torch.int8), torch.where(zero, 1.0, div(amax, 127.0))


@pytest.mark.parametrize("T,K", [(1, 16), (5, 48), (300, 256), (64, 7168), (33, 2000), (2, 32768), (700, 640)])
def test_quantize_rows(T, K):
    x, _, _ = make(T, K, 5)
    x[T // 2] = 0
    q = torch.full((T + 3, K), 77, dtype=torch.int8, device="cuda")
    s = torch.full((T + 3,), -5.0, device="cuda")
    moe.int8_quantize(x, q, s)
    c, sc = codes64(x)
    assert torch.equal(q[:T], c) and torch.equal(s[:T], sc)
    assert bool((q[T:] == 77).all()) and bool((s[T:] == -5).all())
    check_codes(q[:T].float(), s[:T].double()[:, None], x.double(), 0.0, 0.5)


@pytest.mark.parametrize("T,K,k", [(1, 128, 8), (100, 256, 2), (512, 2048, 8), (9, 7168, 32), (3, 64, 40)])
def test_quantize_scatter(T, K, k):
    x, _, _ = make(T, K, 6)
    R = T * k + 5
    g = torch.Generator().manual_seed(7)
    inv = torch.randperm(R, generator=g)[:T * k].int()
    if T * k > 4:
        inv[1], inv[T * k - 2], inv[2] = -1, R, -2147483648    # dropped pairs, entries out of range
    q = torch.full((R, K), 77, dtype=torch.int8, device="cuda")
    s = torch.full((R,), -5.0, device="cuda")
    moe.int8_quantize(x, q, s, inv_perm=inv.cuda(), k=k)
    c, sc = codes64(x)
    want_q, want_s = torch.full_like(q, 77), torch.full_like(s, -5.0)
    at = inv.long()
    ok = (at >= 0) & (at < R)
    rows = (torch.arange(T * k) // k)[ok].cuda()
    want_q[at[ok].cuda()] = c[rows]
    want_s[at[ok].cuda()] = sc[rows]
    assert torch.equal(q, want_q) and torch.equal(s, want_s)


def test_quantize_special_rows():
    x = torch.ones(5, 32, dtype=torch.bfloat16, device="cuda")
    x[0, 3], x[1, 4] = math.nan, math.inf
    x[2] = 2.0 ** -101
    x[3] = 2.0 ** -99
    q, s = torch.empty(5, 32, dtype=torch.int8, device="cuda"), torch.empty(5, device="cuda")
    moe.int8_quantize(x, q, s)
    assert bool(torch.isnan(s[0])) and bool(torch.isinf(s[1])) and bool((q[:3] == 0).all())
    assert s[2] == 1 and bool((q[3:] == 127).all())


def test_empty_calls():
    x = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(128, device="cuda")
    assert moe.moe_rmsnorm_quant(x, w, 1e-6, y=torch.empty_like(x)) == moe.MOE_OK
    assert moe.int8_quantize(x, torch.empty(0, 128, dtype=torch.int8, device="cuda"),
                             torch.empty(0, device="cuda")) == moe.MOE_OK


def test_side_stream_and_capture():
    x, res, w = make(70, 512, 8)
    q, s = torch.empty(70, 512, dtype=torch.int8, device="cuda"), torch.empty(70, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    run = lambda: moe.moe_rmsnorm_quant(x, w, 1e-6, residual=res, q_format="int8", q=q, q_scale=s)  # noqa: E731
    with torch.cuda.stream(side):
        run()
    torch.cuda.synchronize()
    check_rows("int8", False, q, s, reference(x, res, w, 1e-6)[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    x.copy_(make(70, 512, 9)[0])
    graph.replay()
    torch.cuda.synchronize()
    check_rows("int8", False, q, s, reference(x, res, w, 1e-6)[1])


@pytest.mark.parametrize("fmt", ["fp8", "mxfp8", "int8"])
def test_norm_rows_that_are_not_finite(fmt):
    """What a NaN, an infinity and a y beyond fp32 leave in every group of their row."""
    T, H = 5, 512
    x, _, _ = make(T, H, 11)
    res = torch.zeros_like(x)
    w = torch.ones(H, device="cuda")
    x[0, 300] = math.nan
    x[1, 300] = -math.inf
    x[2, 300] = res[2, 300] = 3e38            # an infinity as bf16(x + residual)
    w[130] = 3.4e38
    x[3] = 1.0
    x[3, 130] = 64.0
    x[4] = 1.0
    x[4, 130] = 0.0
    q, s = outputs(T, H, fmt, False)
    y = torch.empty_like(x)
    moe.moe_rmsnorm_quant(x, w, 1e-6, residual=res, y=y, q_format=fmt, q=q[:T], q_scale=s)
    assert bool(torch.isnan(y[0]).all())
    for t in (1, 2):
        assert bool(torch.isnan(y[t, 300])) and bool((torch.cat([y[t, :300], y[t, 301:]]) == 0).all())
    assert bool(torch.isinf(y[3, 130])) and bool(torch.isfinite(y[3, 131:]).all())
    if fmt == "int8":
        assert bool(torch.isnan(s[:3]).all()) and bool(torch.isinf(s[3])) and bool((q[:4] == 0).all())
        return
    v = q[:T].view(torch.float8_e4m3fn).float()
    blk = 128 if fmt == "fp8" else 32
    hit, over = 300 // blk, 130 // blk
    bad = torch.isnan(s) if fmt == "fp8" else s == 255
    clean = s == 1 if fmt == "fp8" else s == 0
    want = torch.zeros_like(bad)
    want[0], want[1, hit], want[2, hit] = True, True, True
    if fmt == "mxfp8":
        want[3, over] = True
    else:
        assert bool(torch.isinf(s[3, over]))
    assert torch.equal(bad, want)
    for t in (1, 2):
        others = torch.arange(H // blk, device="cuda") != hit
        assert bool(clean[t][others].all())
        assert bool((v[t].view(-1, blk)[others] == 0).all())
