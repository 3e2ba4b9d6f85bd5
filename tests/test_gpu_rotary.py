"""pa_rotate_and_cache against the oracle: every product and sum is rounded to
fp32 by itself and the result once to the stored type, so the bits are those of
the oracle computed in fp32; and the values are within the bounds that those
roundings give of the oracle in fp64."""
import numpy as np
import pytest
import torch

from oracle import fp8, int8
from oracle.rotary import pair_dims, rotate
from paged_kv_cache_361_b200 import PagedKVCache, binding as B

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}


@pytest.fixture(autouse=True)
def _clean_error_word():
    B.pa_get_device_error()
    yield


def _bits(t):
    return t.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def _as_stored(y32, dtype, scale):
    """fp32 numpy rows as the cache holds them."""
    if dtype == "e4m3":
        return torch.from_numpy(fp8.quantize(y32, scale))
    if dtype == "int8":
        return torch.from_numpy(int8.quantize(y32, scale))
    return torch.from_numpy(y32).to(DT[dtype])


def _case(seed, tokens, hq, hkv, D, bs, dtype, rd, fused=True, nb=None, max_pos=5000):
    g = torch.Generator().manual_seed(seed)
    dt = B.input_dtype(DT[dtype])
    qkv = torch.randn(tokens, (hq + 2 * hkv) * D, generator=g).to(dt)
    parts = [p.unflatten(1, (-1, D)) for p in qkv.cuda().split([hq * D, hkv * D, hkv * D], 1)]
    if not fused:
        parts = [p.contiguous() for p in parts]
    nb = nb or -(-tokens // bs) + 2
    slots = torch.randperm(nb * bs, generator=g)[:tokens]
    pos = torch.randint(0, max_pos, (tokens,), generator=g, dtype=torch.int32)
    kc = torch.zeros(nb, hkv, bs, D, dtype=DT[dtype], device="cuda")
    kc.view(torch.uint8).fill_(0x5A)
    vc = kc.clone()
    if dtype in ("e4m3", "int8"):
        B.set_kv_scales(kc, vc, 0.013, 0.021)
    return qkv, parts, slots, pos, kc, vc


def _check(qkv, slots, pos, table, kc, vc, q_out, hq, hkv, dtype, interleaved, cached=None):
    T, rd, D = len(pos), table.shape[1], kc.shape[3]
    cos, sin = (x.numpy() for x in table[pos.long()].split(rd // 2, 1))
    x = qkv.float().numpy().reshape(T, -1, D)
    y32 = rotate(x[:, :hq + hkv], cos, sin, interleaved)
    y64 = rotate(x[:, :hq + hkv].astype(np.float64), cos.astype(np.float64), sin.astype(np.float64), interleaved)
    a_dims, b_dims = pair_dims(rd, interleaved)
    mag = np.abs(y64)
    for u, w in ((a_dims, b_dims), (b_dims, a_dims)):
        mag[..., u] = np.abs(x[:, :hq + hkv][..., u] * cos[:, None]) + np.abs(x[:, :hq + hkv][..., w] * sin[:, None])
    # each product and the sum rounded by half a step, 2^-24, of at most |a cos| + |b sin|
    # (the sum's by that of a value 2^-24 larger: the third 2^-24 covers it)
    assert (np.abs(y32 - y64) <= 3 * 2.0 ** -24 * mag).all()
    if q_out is not None:
        assert torch.equal(_bits(q_out.cpu()), _bits(torch.from_numpy(y32[:, :hq]).to(q_out.dtype)))
    cached = torch.ones(T, dtype=torch.bool) if cached is None else cached
    for pool, rows, scale in ((kc, y32[:, hq:], 0.013), (vc, np.ascontiguousarray(x[:, hq + hkv:]), 0.021)):
        exp = torch.full(pool.shape, 0, dtype=pool.dtype)
        exp.view(torch.uint8).fill_(0x5A)            # what no token names stays as it was
        flat = _bits(exp).transpose(1, 2).reshape(-1, hkv, D).clone()
        flat[slots[cached]] = _bits(_as_stored(np.ascontiguousarray(rows), dtype, scale))[cached]
        got = _bits(pool.cpu()).transpose(1, 2).reshape(-1, hkv, D)
        assert torch.equal(got, flat)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "e4m3", "int8"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rd", [(128, 128), (128, 48), (128, 16), (64, 64), (64, 32)])
def test_rotate_matches_the_oracle_bit_for_bit(dtype, interleaved, D, rd):
    for tokens, hq, hkv, bs, fused in ((1, 1, 1, 1, True), (7, 8, 2, 16, True), (37, 3, 3, 4, False), (130, 16, 8, 32, True)):
        qkv, (q, k, v), slots, pos, kc, vc = _case(tokens * D + rd, tokens, hq, hkv, D, bs, dtype, rd, fused)
        table = B.rotary_table(5000, rd)
        q_out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
        B.pa_rotate_and_cache(q, k, v, pos.cuda(), table, slots.cuda(), kc, vc, q_out, interleaved=interleaved)
        assert B.pa_get_device_error()[0] == B.PA_OK
        _check(qkv, slots, pos, table.cpu(), kc, vc, q_out, hq, hkv, dtype, interleaved)


def test_without_q_in_place_and_empty():
    qkv, (q, k, v), slots, pos, kc, vc = _case(3, 21, 4, 2, 64, 8, "bf16", 64, fused=False)
    table = B.rotary_table(5000, 64)
    B.pa_rotate_and_cache(None, k, v, pos.cuda(), table, slots.cuda(), kc, vc, None)
    _check(qkv, slots, pos, table.cpu(), kc, vc, None, 4, 2, "bf16", False)
    before = q.clone()
    B.pa_rotate_and_cache(q, k, v, pos.cuda(), table, slots.cuda(), kc, vc, q)       # q in its own place
    _check(qkv, slots, pos, table.cpu(), kc, vc, q, 4, 2, "bf16", False)
    assert not torch.equal(before, q)
    empty = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    B.pa_rotate_and_cache(None, empty, empty, pos[:0].cuda(), table, slots[:0].cuda(), kc, vc, None)
    assert B.pa_get_device_error()[0] == B.PA_OK


def test_left_out_tokens_and_bad_indexes():
    """A slot of -1 keeps the token out of the cache but rotates its q; a slot
    outside the pool does the same and is recorded; a position outside the table
    leaves the whole token out and is recorded."""
    qkv, (q, k, v), slots, pos, kc, vc = _case(5, 9, 4, 2, 128, 16, "bf16", 128)
    table = B.rotary_table(5000, 128)
    nslots = kc.shape[0] * 16
    bad = slots.clone()
    bad[2] = -1
    q_out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
    B.pa_rotate_and_cache(q, k, v, pos.cuda(), table, bad.cuda(), kc, vc, q_out)
    assert B.pa_get_device_error()[0] == B.PA_OK
    cached = torch.ones(9, dtype=torch.bool)
    cached[2] = False
    _check(qkv, slots, pos, table.cpu(), kc, vc, q_out, 4, 2, "bf16", False, cached)

    for value in (nslots, -2, 1 << 40):
        qkv, (q, k, v), slots, pos, kc, vc = _case(6, 9, 4, 2, 128, 16, "bf16", 128)
        bad = slots.clone()
        bad[2] = value
        B.pa_rotate_and_cache(q, k, v, pos.cuda(), table, bad.cuda(), kc, vc, q_out)
        assert B.pa_get_device_error()[0] == B.PA_ERR_DEVICE_BOUNDS
        _check(qkv, slots, pos, table.cpu(), kc, vc, q_out, 4, 2, "bf16", False, cached)

    for value in (5000, -1, 2 ** 31 - 1):
        qkv, (q, k, v), slots, pos, kc, vc = _case(7, 9, 4, 2, 128, 16, "bf16", 128)
        bad = pos.clone()
        bad[2] = value
        q_out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
        B.pa_rotate_and_cache(q, k, v, bad.cuda(), table, slots.cuda(), kc, vc, q_out)
        assert B.pa_get_device_error()[0] == B.PA_ERR_DEVICE_BOUNDS
        assert (q_out[2] == 7.0).all()
        _check(qkv, slots, pos, table.cpu(), kc, vc, None, 4, 2, "bf16", False, cached)


def test_offsets_past_32_bits():
    """A pool of more than 2^31 elements: its last slots are written where they
    belong (5.4 GB per pool, rows read back through 64-bit indexing)."""
    hkv, D, bs = 8, 128, 32
    nb = (1 << 31) // (hkv * D * bs) + 16
    kc = torch.zeros(nb, hkv, bs, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    g = torch.Generator().manual_seed(0)
    k, v = (torch.randn(3, hkv, D, generator=g).bfloat16() for _ in "kv")
    slots = torch.tensor([nb * bs - 1, 0, (nb - 9) * bs + 5])
    pos = torch.tensor([4, 0, 99], dtype=torch.int32)
    table = B.rotary_table(100, D)
    B.pa_rotate_and_cache(None, k.cuda(), v.cuda(), pos.cuda(), table, slots.cuda(), kc, vc, None)
    cos, sin = (x.numpy() for x in table.cpu()[pos.long()].split(D // 2, 1))
    want = torch.from_numpy(rotate(k.float().numpy(), cos, sin, False)).bfloat16()
    for i, s in enumerate(slots.tolist()):
        assert torch.equal(kc[s // bs, :, s % bs].cpu(), want[i])
        assert torch.equal(vc[s // bs, :, s % bs].cpu(), v[i])
    assert int((vc.view(torch.int16)[-16:] != 0).any(-1).sum()) == 2 * hkv


@pytest.mark.parametrize("dtype", ["e4m3", "int8"])
@pytest.mark.parametrize("k_scale,v_scale", [(0.1, 3e-33), (2.0 ** -6, 7.3), (1.7e36, 1e-3)])
def test_codes_at_any_scale(dtype, k_scale, v_scale):
    """Codes bit for bit at scales whose reciprocal is exact, rounded and out of
    the usual range, for values next to and on the borders between codes."""
    g = torch.Generator().manual_seed(2)
    n, hkv, D = 64, 2, 128
    k, v = (torch.randn(n, hkv, D, generator=g) * s * 40 for s in (k_scale, v_scale))
    # half of the values on multiples of half a code's step
    k[::2], v[::2] = ((x[::2] / s * 2).round() / 2 * s for x, s in ((k, k_scale), (v, v_scale)))
    k, v = k.bfloat16(), v.bfloat16()
    k[1, 0, :4] = torch.tensor([float("inf"), -float("inf"), 0.0, -0.0])
    v[1, 0, :4] = torch.tensor([3e38, -3e38, 1e-40, float("inf")])
    kc = torch.zeros(8, hkv, 8, D, dtype=DT[dtype], device="cuda")
    vc = torch.zeros_like(kc)
    B.set_kv_scales(kc, vc, k_scale, v_scale)
    slots, pos = torch.arange(n), torch.zeros(n, dtype=torch.int32)   # position 0: k as it is
    B.pa_rotate_and_cache(None, k.cuda(), v.cuda(), pos.cuda(), B.rotary_table(1, D), slots.cuda(), kc, vc, None)
    for pool, x, scale in ((kc, k, k_scale), (vc, v, v_scale)):
        x32 = x.float().numpy()
        if pool is kc:   # a 1 - b 0 and b 1 + a 0: an infinity's partner is NaN
            with np.errstate(invalid="ignore"):
                x32 = rotate(x32, np.ones((n, D // 2), np.float32), np.zeros((n, D // 2), np.float32), False)
        got = _bits(pool.cpu()).transpose(1, 2).reshape(n, hkv, D)
        want = _as_stored(np.ascontiguousarray(x32), dtype, scale).view(torch.uint8)
        nan = torch.from_numpy(np.isnan(x32))
        assert torch.equal(got[~nan], want[~nan])
        assert ((got[nan] & 0x7F) == (0x7F if dtype == "e4m3" else 0)).all()


def test_wrong_tensors_are_refused():
    qkv, (q, k, v), slots, pos, kc, vc = _case(8, 6, 4, 2, 64, 8, "bf16", 64)
    table = B.rotary_table(100, 64)
    args = dict(q=q, k=k, v=v, positions=pos.cuda() % 100, cos_sin=table, slot_mapping=slots.cuda(), k_cache=kc,
                v_cache=vc, q_out=torch.empty(q.shape, dtype=q.dtype, device="cuda"))
    for kw in (dict(q=q.float()), dict(k=k.cpu()), dict(positions=pos.cuda().long()), dict(slot_mapping=slots.cuda().int()),
               dict(cos_sin=table.double()), dict(v=v[:3]), dict(q_out=None), dict(q=q[:, :, :32]),
               dict(positions=pos.cuda()[:2]), dict(cos_sin=table[:, ::2]),
               dict(k=k[:, :1]), dict(q_out=torch.empty(6, 4, 128, dtype=q.dtype, device="cuda")[..., :64])):
        with pytest.raises((TypeError, ValueError)):
            B.pa_rotate_and_cache(**dict(args, **kw))
    with pytest.raises(B.PagedAttnError) as e:
        B.pa_rotate_and_cache(**dict(args, cos_sin=B.rotary_table(100, 8)))
    assert e.value.status == B.PA_ERR_UNSUPPORTED


def test_captured_and_on_another_stream():
    qkv, (q, k, v), slots, pos, kc, vc = _case(9, 40, 8, 2, 128, 16, "bf16", 128)
    table, pos_d, slots_d = B.rotary_table(5000, 128), pos.cuda(), slots.cuda()
    q_out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        B.pa_rotate_and_cache(q, k, v, pos_d, table, slots_d, kc, vc, q_out)
    for step in range(3):
        pos_new = (pos + step) % 5000
        pos_d.copy_(pos_new)
        graph.replay()
        torch.cuda.synchronize()
        _check(qkv, slots, pos_new, table.cpu(), kc, vc, q_out, 8, 2, "bf16", False)
    kc.view(torch.uint8).fill_(0x5A)
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.default_stream())
        B.pa_rotate_and_cache(q, k, v, pos_d, table, slots_d, kc, vc, q_out)
    side.synchronize()
    _check(qkv, slots, pos_new, table.cpu(), kc, vc, q_out, 8, 2, "bf16", False)


def test_append_rotated_then_decode():
    """The cache's own path: prompts and steps appended with their rotation,
    decoded, against attention over rows rotated by the oracle."""
    from oracle.attention import decode_attention
    hq, hkv, D = 8, 2, 64
    g = torch.Generator().manual_seed(11)
    cache = PagedKVCache(20, hkv, 16, D, torch.bfloat16, "cuda", fill=float("nan"))
    table = B.rotary_table(200, D)
    hist = {0: ([], []), 1: ([], [])}
    rot = lambda x, p: rotate(x.float().numpy(), *(t.numpy() for t in table.cpu()[p].split(D // 2, 1)), False)
    for counts in ([21, 40], [1, 1], [3, 1], [1, 1]):
        T = sum(counts)
        q, k, v = (torch.randn(T, h, D, generator=g).bfloat16() for h in (hq, hkv, hkv))
        first = [len(hist[s][0]) for s in (0, 1)]
        p = torch.cat([torch.arange(f, f + c) for f, c in zip(first, counts)])
        q_rot = cache.append_rotated([0, 1], counts, q.cuda(), k.cuda(), v.cuda(), table)
        kr = torch.from_numpy(rot(k, p)).bfloat16()
        assert torch.equal(q_rot.cpu(), torch.from_numpy(rot(q, p)).bfloat16())
        for s, (a, b) in enumerate(((0, counts[0]), (counts[0], T))):
            hist[s][0].extend(kr[a:b])
            hist[s][1].extend(v[a:b])
        last = torch.tensor([counts[0] - 1, T - 1])
        out = cache.decode([0, 1], q_rot[last.cuda()].contiguous()).cpu()
        for s in (0, 1):
            ref = decode_attention(q_rot[last[s]].cpu(), torch.stack(hist[s][0]), torch.stack(hist[s][1]), D ** -0.5)
            assert np.abs(out[s].double().numpy() - ref).max() <= 4e-3
    assert B.pa_get_device_error()[0] == B.PA_OK
