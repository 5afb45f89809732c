"""Refusals of the scored router, the RMS norm, the int8 quantiser and the
int8 GEMM: wrong arguments are turned down before any launch, without a GPU."""
import os

import pytest
import torch

import fp8_block_scaled_route_b200 as moe

FAKE = 1 << 20  # an aligned address never dereferenced: validation fails first
INVALID, UNSUPPORTED = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from fp8_block_scaled_route_b200 import build
    build.build()
    moe.lib()


def _score(T=8, E=64, k=4, logits=FAKE, ids=FAKE, w=FAKE, logits_dtype="float32", **how):
    return moe.moe_router_score_topk(logits, ids, w, dims=(T, E, k), logits_dtype=logits_dtype,
                                     stream=0, check=False, **how)


@pytest.mark.parametrize("args,want", [
    (dict(T=-1), INVALID), (dict(k=0), INVALID), (dict(k=65), INVALID), (dict(E=128, k=33), INVALID),
    (dict(E=2048), UNSUPPORTED), (dict(logits_dtype=7), INVALID), (dict(scoring=2), INVALID),
    (dict(n_group=0), INVALID), (dict(n_group=5), INVALID), (dict(n_group=64), INVALID),
    (dict(n_group=4, topk_group=0), INVALID), (dict(n_group=4, topk_group=5), INVALID),
    (dict(group_top=3), INVALID), (dict(n_group=32, topk_group=1, k=3), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(logits=0), INVALID), (dict(ids=0), INVALID),
    (dict(w=0), INVALID), (dict(T=1 << 28, k=32, E=64), UNSUPPORTED), (dict(T=2 ** 31 - 1, k=1), UNSUPPORTED),
    (dict(logits=FAKE + 2), INVALID),
    (dict(ids=FAKE + 1), INVALID), (dict(w=FAKE + 2), INVALID), (dict(bias=FAKE + 2), INVALID),
])
def test_score_refusals(args, want):
    assert _score(**args) == want


def test_score_route_refusals():
    def r(m=FAKE, perm=FAKE, ws=FAKE, ws_bytes=1 << 20, **how):
        return moe.moe_router_score_route(FAKE, FAKE, FAKE, m, perm, None, ws, ws_bytes,
                                          dims=(8, 64, 4), stream=0, check=False, **how)
    assert r(m=0) == INVALID
    assert r(perm=0) == INVALID
    assert r(m=FAKE + 2) == INVALID and r(perm=FAKE + 1) == INVALID
    assert r(ws=0) == INVALID
    assert r(ws=FAKE + 4) == INVALID
    assert r(ws_bytes=64) == INVALID
    assert r(n_group=3) == INVALID


def _norm(T=4, H=256, x=FAKE, weight=FAKE, eps=1e-6, weight_dtype="float32", y=FAKE, **how):
    return moe.moe_rmsnorm_quant(x, weight, eps, y=y, dims=(T, H), weight_dtype=weight_dtype, stream=0,
                                 check=False, **how)


@pytest.mark.parametrize("args,want", [
    (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(H=24), INVALID), (dict(H=32784), UNSUPPORTED),
    (dict(eps=0.0), INVALID), (dict(eps=-1e-6), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=2.0), INVALID), (dict(weight_dtype=3), INVALID), (dict(q_format=4), INVALID),
    (dict(q_format=-1), INVALID), (dict(scale_major=2), INVALID), (dict(y=None), INVALID),
    (dict(x=0), INVALID), (dict(weight=0), INVALID), (dict(x=FAKE + 8), INVALID),
    (dict(y=FAKE + 2), INVALID), (dict(residual_out=FAKE), INVALID),
    (dict(residual=FAKE + 8), INVALID), (dict(weight=FAKE + 4), INVALID),
    (dict(q_format="fp8", q=FAKE, q_scale=FAKE, H=192), INVALID),
    (dict(q_format="mxfp8", q=FAKE, q_scale=FAKE, H=32), INVALID),
    (dict(q_format="int8", q=FAKE), INVALID), (dict(q_format="int8", q_scale=FAKE), INVALID),
    (dict(q_format="int8", q=FAKE + 8, q_scale=FAKE), INVALID),
    (dict(q_format="int8", q=FAKE, q_scale=FAKE + 2), INVALID),
])
def test_norm_refusals(args, want):
    assert _norm(**args) == want


@pytest.mark.parametrize("args,want", [
    (dict(T=-1), INVALID), (dict(K=0), INVALID), (dict(K=24), INVALID), (dict(K=32784), UNSUPPORTED),
    (dict(k=0), INVALID), (dict(k=2), INVALID), (dict(R=3), INVALID), (dict(x=0), INVALID),
    (dict(q=0), INVALID), (dict(s=0), INVALID), (dict(x=FAKE + 2), INVALID), (dict(q=FAKE + 8), INVALID),
    (dict(R=-1), INVALID), (dict(s=FAKE + 2), INVALID),
])
def test_quantize_refusals(args, want):
    a = dict(T=4, K=64, k=1, R=4, x=FAKE, q=FAKE, s=FAKE) | args
    assert moe.int8_quantize(a["x"], a["q"], a["s"], k=a["k"], dims=(a["T"], a["K"], a["R"]), stream=0,
                             check=False) == want


@pytest.mark.parametrize("args,want", [
    (dict(R=-1), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(K=40), INVALID),
    (dict(E=0), INVALID), (dict(E=2, m=None), INVALID), (dict(E=2048), UNSUPPORTED),
    (dict(K=131072), UNSUPPORTED), (dict(N=33, gated=True), INVALID), (dict(od=2), INVALID),
    (dict(E=1024, N=1 << 21), UNSUPPORTED), (dict(a=0), INVALID), (dict(b=0), INVALID),
    (dict(sa=0), INVALID), (dict(sb=0), INVALID), (dict(out=0), INVALID), (dict(a=FAKE + 8), INVALID),
    (dict(b=FAKE + 4), INVALID), (dict(out=FAKE + 2), INVALID), (dict(sa=FAKE + 2), INVALID),
    (dict(sb=FAKE + 1), INVALID), (dict(m=FAKE + 2), INVALID),
])
def test_gemm_refusals(args, want):
    c = dict(R=8, N=32, K=64, E=1, m=FAKE, gated=False, od="bfloat16", a=FAKE, b=FAKE, sa=FAKE, sb=FAKE,
             out=FAKE) | args
    assert moe.int8_moe_gemm(c["a"], c["b"], c["sa"], c["sb"], c["out"], m_indptr=c["m"],
                             is_gated=c["gated"], dims=(c["R"], c["N"], c["K"], c["E"]),
                             out_dtype=c["od"], stream=0, check=False) == want


def test_refusal_raises():
    with pytest.raises(moe.MoEError) as e:
        moe.int8_moe_gemm(FAKE, FAKE, FAKE, FAKE, FAKE, m_indptr=FAKE, dims=(8, 32, 40, 1), stream=0)
    assert e.value.status == INVALID


def test_tensor_checks():
    """Tensors that the C entry would misread are refused by the binding."""
    bf, i8 = torch.bfloat16, torch.int8
    x, w = torch.zeros(4, 128, dtype=bf), torch.ones(128)
    y = torch.empty_like(x)
    for bad in (dict(x=x.float()), dict(x=torch.zeros(128, 4, dtype=bf).t()), dict(weight=w.half()),
                dict(y=torch.empty(3, 128, dtype=bf)), dict(residual=x.float()),
                dict(y=torch.empty(8, 128, dtype=bf)[::2])):
        a = dict(x=x, weight=w, y=y, residual=None) | bad
        with pytest.raises(ValueError):
            moe.moe_rmsnorm_quant(a["x"], a["weight"], 1e-6, residual=a["residual"], y=a["y"])
    with pytest.raises(ValueError):    # scales laid out for the other major
        moe.moe_rmsnorm_quant(x, w, 1e-6, q_format="fp8", q=torch.empty(4, 128, dtype=torch.uint8),
                              q_scale=torch.empty(4, 1), scale_major="MN")
    q, s = torch.empty(4, 128, dtype=i8), torch.empty(4)
    with pytest.raises(ValueError):
        moe.int8_quantize(x, q, s, inv_perm=torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError):
        moe.int8_quantize(x, q[:, :64], s)
    a, b = torch.zeros(4, 64, dtype=i8), torch.zeros(2, 32, 64, dtype=i8)
    sa, sb, m = torch.ones(4), torch.ones(2, 32), torch.zeros(3, dtype=torch.int32)
    out = torch.empty(4, 32, dtype=bf)
    for bad in (dict(a=a.to(torch.uint8)), dict(b=b[:, :, :32]), dict(sa=sa[:3]), dict(sb=sb[:1]),
                dict(m=m[:2]), dict(out=out[:, :16]), dict(out=out.half()), dict(m=m.long())):
        c = dict(a=a, b=b, sa=sa, sb=sb, m=m, out=out) | bad
        with pytest.raises(ValueError):
            moe.int8_moe_gemm(c["a"], c["b"], c["sa"], c["sb"], c["out"], m_indptr=c["m"])
    logits, ids, tw = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    for bad in (dict(logits=logits.half()), dict(ids=ids.long()), dict(w=tw[:3]),
                dict(bias=torch.zeros(7)), dict(bias=torch.zeros(8, dtype=bf))):
        c = dict(logits=logits, ids=ids, w=tw, bias=None) | bad
        with pytest.raises(ValueError):
            moe.moe_router_score_topk(c["logits"], c["ids"], c["w"], bias=c["bias"])
    with pytest.raises(ValueError):    # right tensors, wrong machine
        moe.moe_router_score_topk(logits, ids, tw)


def test_every_entry_point_documented():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    readme = open(os.path.join(root, "README.md")).read()
    for name in ("moe_router_score_topk", "moe_router_score_route", "moe_rmsnorm_quant", "int8_quantize",
                 "int8_moe_gemm"):
        assert name in readme


def test_dependent_kernels_read_coherently():
    """A kernel that may be resident before its predecessor has ended must not
    read that one's outputs through the read-only path: neither __ldg nor a
    pointer declared as never written while the kernel runs."""
    root = os.path.dirname(os.path.abspath(moe.__file__))
    seen = 0
    for name in sorted(os.listdir(os.path.join(root, "csrc"))):
        text = open(os.path.join(root, "csrc", name)).read()
        code = "\n".join(line.split("//")[0] for line in text.splitlines())
        if name.endswith(".cu") and "pdl_wait(" in code:
            seen += 1
            for word in ("__ldg(", "__restrict__", "ld.global.nc"):
                assert word not in code, f"{name}: {word}"
    assert seen >= 3


@pytest.mark.parametrize("shape", [(64,), (32, 1, 1, 64), ()])
def test_gemm_weights_have_two_or_three_dimensions(shape):
    """Weights of another rank are named as what is wrong: a vector of K codes
    would be read as K rows of them."""
    a, b = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(shape, dtype=torch.int8)
    n = shape[0] if shape else 64
    with pytest.raises(ValueError, match="b has"):
        moe.int8_moe_gemm(a, b, torch.ones(4), torch.ones(n), torch.empty(4, n))


@pytest.mark.parametrize("how", [
    dict(residual=FAKE, residual_out=3 * FAKE, y=3 * FAKE), dict(residual=2 * FAKE, residual_out=FAKE, y=FAKE),
    dict(y=3 * FAKE, q_format="int8", q=3 * FAKE, q_scale=4 * FAKE),
    dict(y=3 * FAKE, q_format="int8", q=FAKE, q_scale=4 * FAKE),
    dict(residual=2 * FAKE, residual_out=3 * FAKE, y=4 * FAKE, q_format="fp8", q=3 * FAKE, q_scale=5 * FAKE),
    dict(residual=2 * FAKE, y=4 * FAKE, q_format="mxfp8", q=2 * FAKE, q_scale=5 * FAKE),
])
def test_norm_refuses_one_buffer_for_two_outputs(how):
    """Two outputs in one buffer, or 8-bit rows over the rows they come from:
    each row would overwrite what another still needs."""
    assert _norm(weight=9 * FAKE, **how) == INVALID


def test_bf16_logits_are_aligned_to_their_size():
    assert _score(logits=FAKE + 1, logits_dtype="bfloat16") == INVALID
    assert _score(logits=FAKE + 2, logits_dtype="bfloat16", ids=FAKE + 2) == INVALID
