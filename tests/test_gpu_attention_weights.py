"""Weights of pa_decode_multi and pa_prefill_window at the ends of their range, in
every form of the kernels, against the oracle in 64 bits.

Bounds of the values. Where weights are rounded to f16 (11 bits) they are packed as 2^7 to 2^15
at the largest, so a weight is off by 2^-11 of itself or by half of f16's least
step, 2^-25, which is 2^-32 of the largest: over n keys by n 2^-32 max|V| together,
the denominator being the largest weight at least. Scores are sums of D products in
fp32, off by at most D 2^-24 sum|q_i k_i| scale: 2e-4 for a sum of 26 (the first
key's 17.7 and the other dims' 7), so that a weight over the denominator is off by
2^-12 of itself. V as f16 is off by 2^-25 at most below 2^-14, and the result is
rounded to bf16 (half a step, 2^-8 of itself).
"""
import numpy as np
import pytest
import torch

from oracle import fp8, int8
from oracle.options import options_attention
from paged_kv_cache_361_b200 import binding as B

pytestmark = pytest.mark.gpu

W = 2.0 ** -11 + 2.0 ** -12
SCALE = {"bf16": (1.0, 1.0), "e4m3": (0.011, 0.017), "int8": (0.031, 0.027)}
DT = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}


@pytest.fixture(autouse=True)
def _clean_error_word():
    B.pa_get_device_error()
    yield


def _paged(rows, dtype, scale):
    """[L][1][D] fp32 rows as a pool of 32-token blocks in order, and their stored values."""
    if dtype == "bf16":
        stored = rows.bfloat16()
        value = stored.double().numpy()
    else:
        q = fp8 if dtype == "e4m3" else int8
        codes = q.quantize(rows.numpy(), scale)
        stored, value = torch.from_numpy(codes).view(DT[dtype]), q.dequantize(codes, scale)
    L, hkv, D = rows.shape
    raw = stored.view(torch.int16 if dtype == "bf16" else torch.uint8)
    pool = torch.zeros(-(-L // 32) * 32, hkv, D, dtype=raw.dtype)
    pool[:L] = raw
    return pool.view(-1, 32, hkv, D).transpose(1, 2).contiguous().view(DT[dtype]).cuda(), value


def _call(kc, vc, q, L, P=None, **rule):
    """P: partition_tokens of pa_decode_multi, None: pa_prefill_window."""
    n, hq, D = q.shape
    tables = torch.arange(kc.shape[0], dtype=torch.int32, device="cuda")[None]
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    out = torch.empty(n, hq, D, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(n, hq, device="cuda")
    args = (q.cuda(), cu, kc, vc, tables, lens, D ** -0.5, out, n, L)
    if P is None:
        B.pa_prefill_window(*args, lse=lse, **rule)
    else:
        need = B.pa_decode_multi_workspace_bytes(n, 1, n, hq, kc.shape[1], D, L, rule.get("window", 0), P)
        B.pa_decode_multi(*args, lse=lse, partition_tokens=P, **rule,
                          workspace=torch.full((need,), 255, dtype=torch.uint8, device="cuda"))
    assert B.pa_get_device_error()[0] == B.PA_OK
    return out.cpu(), lse.cpu()


# (new tokens, query heads, partition_tokens): rows on mma.sync, with four, two and one
# state a row on tcgen05, and pa_prefill_window
FORMS = [(1, 1, 0), (2, 4, -1), (3, 4, 0), (5, 8, 0), (5, 8, -1), (16, 8, 0), (17, 4, None)]


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 64), ("e4m3", 128), ("int8", 64)])
@pytest.mark.parametrize("n,hq,P", FORMS)
@pytest.mark.parametrize("spread", [False, True])
def test_a_first_key_that_outweighs_a_long_tail(dtype, D, n, hq, P, spread):
    """The first key has 99.9 % of the weight and a V of 0: the result is that of the
    tail, 33000 keys of weights next to 2^-25.5 of the first's."""
    L = 33001
    g = torch.Generator().manual_seed(n + hq + D)
    q = torch.randn(n, hq, D, generator=g)
    q[..., 0] = 64.0
    K = torch.randn(L, 1, D, generator=g) * (1.0 if spread else 0.0)
    K[:, :, 0] = 0.0
    K[0] = 0.0
    K[0, 0, 0] = 25.5 * np.log(2.0) / 64.0 * D ** 0.5
    V = 1.0 + 0.25 * torch.randn(L, 1, D, generator=g)
    V[0] = 0.0
    q = q.bfloat16()
    (kc, kv), (vc, vv) = _paged(K, dtype, SCALE[dtype][0]), _paged(V, dtype, SCALE[dtype][1])
    if dtype != "bf16":
        B.set_kv_scales(kc, vc, *SCALE[dtype])
    out, lse = _call(kc, vc, q, L, P)
    ref, want, size = options_attention(q, kv, vv, D ** -0.5)
    tol = 2.0 ** -8 * np.abs(ref) + (1 + 2.0 ** -8) * (W * size + L * 2.0 ** -32 * np.abs(vv).max()) + 2.0 ** -24
    err = np.abs(out.double().numpy() - ref)
    assert (err <= tol).all(), float((err - tol).max())
    assert (np.abs(lse.double().numpy() - want) <= 2.0 ** -12 + 2.0 ** -23 * np.abs(want)).all()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,hq,P", FORMS + [(2, 4, 64), (5, 8, 128), (2, 4, 512), (5, 8, 2048)])
def test_a_query_of_nan_gives_nan(dtype, n, hq, P):
    """All scores of a row are NaN then: its result is NaN, as by the formula, not
    that of a row without keys; the other rows keep theirs bit for bit."""
    L, D = 5000, 64
    g = torch.Generator().manual_seed(n)
    q = torch.randn(n, hq, D, generator=g).bfloat16()
    kc, _ = _paged(torch.randn(L, 1, D, generator=g), dtype, SCALE[dtype][0])
    vc, _ = _paged(torch.randn(L, 1, D, generator=g), dtype, SCALE[dtype][1])
    if dtype != "bf16":
        B.set_kv_scales(kc, vc, *SCALE[dtype])
    for sinks in (None, torch.zeros(hq, device="cuda")):
        out, lse = _call(kc, vc, q, L, P, sinks=sinks)
        bad = q.clone()
        bad[n - 1, hq // 2] = float("nan")
        got, got_lse = _call(kc, vc, bad, L, P, sinks=sinks)
        hit = torch.zeros(n, hq, dtype=torch.bool)
        hit[n - 1, hq // 2] = True
        assert got[hit].isnan().all() and got_lse[hit].isnan().all()
        assert torch.equal(got[~hit], out[~hit]) and torch.equal(got_lse[~hit], lse[~hit])


@pytest.mark.parametrize("dtype", ["e4m3", "int8"])
@pytest.mark.parametrize("n,hq,P", FORMS + [(2, 4, 64), (5, 8, 512)])
def test_a_small_v_scale_keeps_its_bits(dtype, n, hq, P):
    """A v_scale of 2^-126, fp32's least normal number: the results, means of 4999
    values of 2^-120 or so, are normal numbers again, and v_scale being a power of
    two they are those of v_scale 1 times 2^-126 bit for bit."""
    L, D = 4999, 64
    g = torch.Generator().manual_seed(n)
    q = torch.randn(n, hq, D, generator=g).bfloat16()
    k_scale = SCALE[dtype][0]
    kc, _ = _paged(torch.randn(L, 1, D, generator=g), dtype, k_scale)
    vc, _ = _paged(80.0 + 20.0 * torch.rand(L, 1, D, generator=g), dtype, 1.0)
    got = []
    for v_scale in (1.0, 2.0 ** -126):
        B.set_kv_scales(kc, vc, k_scale, v_scale)
        got.append(_call(kc, vc, q, L, P))
    assert torch.equal(got[0][0].double() * 2.0 ** -126, got[1][0].double())
    assert torch.equal(got[0][1], got[1][1])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,hq,P", [(2, 4, 64), (3, 4, 0), (5, 8, 0), (5, 8, 128), (16, 8, 0), (17, 4, None), (40, 1, None)])
@pytest.mark.parametrize("window", [0, 45])
def test_capped_bits_do_not_depend_on_bytes_that_no_row_sees(n, hq, P, window, D):
    """Scores small beside the cap; the slots behind the last token, and those before
    the first window in a block that it starts in, hold zeros, then large values,
    infinities and NaN."""
    L = 331
    g = torch.Generator().manual_seed(n + D)
    q = torch.randn(n, hq, D, generator=g).bfloat16()
    kc, _ = _paged(torch.randn(L, 1, D, generator=g), "bf16", 1.0)
    vc, _ = _paged(torch.randn(L, 1, D, generator=g), "bf16", 1.0)
    first = max(0, L - n - window + 1) if window else 0
    got = []
    for filler in (0.0, 30.0, 3000.0, float("inf"), float("nan")):
        for pool in (kc, vc):
            flat = pool.transpose(1, 2).reshape(-1, 1, D)
            flat[:first] = filler
            flat[L:] = filler
            pool.copy_(flat.view(-1, 32, 1, D).transpose(1, 2))
        got.append(_call(kc, vc, q, L, P, window=window, softcap=50.0))
    for out, lse in got[1:]:
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])
