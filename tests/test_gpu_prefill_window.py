"""pa_prefill_window against the oracle in 64 bits, and PagedKVCache.attend.

Bounds as in test_gpu_decode_multi.py; the weights and V enter the product as
f16 over every cache (half a step, 2^-11; V exactly, but for values below 2^-14,
which move by 2^-25 at most): W = 2^-11 + 2^-12, and 2^-24 beside it."""
import numpy as np
import pytest
import torch

from oracle.options import options_attention_masked
from oracle.rotary import rotate
from paged_kv_cache_361_b200 import PagedKVCache, binding as B
from tests.test_gpu_decode_multi import LSE, Batch, _sinks

pytestmark = pytest.mark.gpu

W = 2.0 ** -11 + 2.0 ** -12


@pytest.fixture(autouse=True)
def _clean_error_word():
    B.pa_get_device_error()
    yield


def _run(b, counts, hq, window=0, cap=0.0, sinks=None, tables=None, want_lse=True, max_q=None):
    T, D = sum(counts), b.kc.shape[3]
    q = torch.randn(T, hq, D, generator=b.g).bfloat16()
    out = torch.full((T, hq, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, hq), float("nan"), device="cuda") if want_lse else None
    cu = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32).cuda()
    B.pa_prefill_window(q.cuda(), cu, b.kc, b.vc, (b.tables if tables is None else tables).cuda(),
                        torch.tensor(b.lens, dtype=torch.int32).cuda(), D ** -0.5, out, max(counts) if max_q is None else max_q,
                        max(b.lens), window=window, softcap=cap, sinks=None if sinks is None else sinks.cuda(), lse=lse)
    torch.cuda.synchronize()
    return q, out.cpu(), None if lse is None else lse.cpu()


def _check_rows(q, got, lse, K, V, window, cap, sinks):
    ref, want, size = options_attention_masked(q, K, V, q.shape[2] ** -0.5, window, cap, sinks)
    got = got.double().numpy()
    tol = 2.0 ** -8 * np.abs(ref) + W * (1 + 2.0 ** -8) * size + 2.0 ** -24
    assert (np.abs(got - ref) <= tol).all(), float((np.abs(got - ref) - tol).max())
    if lse is not None:
        assert (np.abs(lse.double().numpy() - want) <= LSE + 2.0 ** -23 * np.abs(want)).all()


def _check(b, counts, q, out, lse, window=0, cap=0.0, sinks=None):
    at = 0
    for i, n in enumerate(counts):
        s = slice(at, at + n)
        _check_rows(q[s], out[s], None if lse is None else lse[s], b.rows[0][i], b.rows[1][i], window, cap,
                    None if sinks is None else sinks.double().numpy())
        at += n


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("bs", [8, 32])
def test_shapes(dtype, D, G, bs):
    """Prompts and chunks around tiles, chunks and blocks, packed at odd lengths."""
    lens = [1, 63, 64, 129, 300, 513]
    b = Batch(lens, 2, D, bs, dtype, seed=D + G + bs)
    for counts, window, cap, sink in (([1, 63, 64, 129, 300, 513], 0, 0.0, True), ([1, 5, 64, 40, 257, 130], 100, 0.0, False),
                                      ([0, 63, 1, 129, 33, 200], 37, 30.0, True), ([1, 63, 64, 129, 300, 513], 130, 50.0, True)):
        sinks = _sinks(2 * G) if sink else None
        _check(b, counts, *_run(b, counts, 2 * G, window, cap, sinks), window, cap, sinks)
    assert B.pa_get_device_error()[0] == B.PA_OK


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 128, 191, 400, 700, 701, 10 ** 6])
def test_windows(dtype, D, window):
    """Windows of one key, around chunks and query tiles, of the context and past
    it; blocks wholly before every window are gone (table entries -1, bytes NaN)."""
    lens = [700, 64, 333]
    for counts in ([700, 64, 333], [150, 3, 90]):
        b = Batch(lens, 2, D, 16, dtype, seed=window % 97 + D)
        tables = b.tables.clone()
        for i, (L, n) in enumerate(zip(lens, counts)):
            for e in range(max(0, L - n - window + 1) // 16):
                for pool in (b.kc, b.vc):
                    pool.view(torch.uint8)[tables[i, e]] = 0xFF if dtype == "bf16" else 0x7F
                tables[i, e] = -1
        for G in (1, 4):
            _check(b, counts, *_run(b, counts, 2 * G, window, 0.0, None, tables=tables), window)
        assert B.pa_get_device_error()[0] == B.PA_OK


def test_plain_call_agrees_with_pa_prefill():
    """Without options it is pa_prefill rounded to bf16: the two differ by their
    roundings alone."""
    b = Batch([500, 77], 2, 128, 16, "bf16", seed=4)
    q, out, _ = _run(b, [400, 77], 8, want_lse=False)
    full = torch.empty(477, 8, 128, device="cuda")
    B.pa_prefill(q.cuda(), torch.tensor([0, 400, 477], dtype=torch.int32).cuda(), b.kc, b.vc, b.tables.cuda(),
                 torch.tensor([500, 77], dtype=torch.int32).cuda(), 128 ** -0.5, full, 400, 500)
    assert ((out.float() - full.cpu()).abs() <= 2.0 ** -8 * full.cpu().abs() + 2.0 ** -20).all()


def test_sinks_of_every_size_and_growing_scores():
    b = Batch([300], 2, 128, 16, "bf16")
    sinks = torch.tensor([float("-inf"), 1e4, -1e4, 0.0, 80.0, -80.0, 3.0, float("-inf")])
    _check(b, [300], *_run(b, [300], 8, 90, 0.0, sinks), 90, 0.0, sinks)
    # every key outweighs those before it: the running maximum moves in each chunk
    ramp = torch.linspace(-6, 6, 300)[:, None, None].expand(300, 2, 128).bfloat16()
    t = torch.arange(300)
    b.kc[b.tables[0].long()[t // 16].cuda(), :, (t % 16).cuda()] = ramp.cuda()
    b.rows[0][0] = ramp.double().numpy()
    q = torch.ones(300, 4, 128).bfloat16()
    for window, cap in ((0, 0.0), (70, 0.0), (0, 20.0), (70, 20.0)):
        out, lse = torch.empty(300, 4, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(300, 4, device="cuda")
        B.pa_prefill_window(q.cuda(), torch.tensor([0, 300], dtype=torch.int32).cuda(), b.kc, b.vc, b.tables.cuda(),
                            torch.tensor([300], dtype=torch.int32).cuda(), 128 ** -0.5, out, 300, 300, window=window,
                            softcap=cap, lse=lse)
        _check(b, [300], q, out.cpu(), lse.cpu(), window, cap)


@pytest.mark.parametrize("cap", [2.0 ** -40, 0.01, 1.5, 5.0, 6.5, 1000.0, 2.0 ** 40])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_caps_of_every_size(cap, dtype):
    """From caps that flatten every score, past those where rows are on both
    sides of the polynomial's range, to one that changes nothing much."""
    b = Batch([200, 90], 2, 128, 16, dtype, seed=8)
    _check(b, [200, 40], *_run(b, [200, 40], 8, 0, cap), 0, cap)
    b.check([5, 16], *b.run([5, 16], 8, 70, cap), 70, cap)
    b.check([1, 2], *b.run([1, 2], 8, 70, cap), 70, cap)


@pytest.mark.parametrize("cap", [5.0, 30.0, 50.0])
@pytest.mark.parametrize("n", [1, 8, 40])
def test_a_capped_score_alone(n, cap):
    """One key in the window: the log-sum-exp is its capped score, small ones too.
    q.k are whole numbers and the scale is 1/8, so s is exact. s / cap takes three
    roundings of 2^-24, tanh six more and a fit within 3e-8 (from 0.5 on: within
    2^-22 + 2^-23 of 0.46 or more, and its argument's roundings, half as much again),
    cap log2 e and ln 2 three: under 2^-20 of the value. The weight of the key,
    2^(x - m) with x and m two roundings apart, and its logarithm: under 2^-22."""
    g = torch.Generator().manual_seed(n)
    ints = lambda *s: torch.randint(-3, 4, s, generator=g).float()
    cache = PagedKVCache(40, 2, 16, 64, torch.bfloat16, "cuda", fill=float("nan"))
    L = [150, 300, n]
    q, ks = ints(3 * n, 8, 64), [ints(x, 2, 64) for x in L]
    for s, k in enumerate(ks):
        cache.add_sequence(s, k.bfloat16().cuda(), torch.randn(*k.shape, generator=g).bfloat16().cuda())
    lse = torch.empty(3 * n, 8, device="cuda")
    cache.attend([0, 1, 2], [n] * 3, q.bfloat16().cuda(), window=1, softcap=cap, lse=lse)
    k = torch.cat([k[-n:] for k in ks]).double().repeat_interleave(4, 1)
    want = cap * torch.tanh((q.double() * k).sum(2) / 8 / cap)
    assert ((lse.cpu().double() - want).abs() <= 2.0 ** -20 * want.abs() + 2.0 ** -22).all()


def test_rows_of_no_sequence_stay_and_bad_rows_are_left_out():
    b = Batch([150, 60], 2, 64, 16, "bf16")
    q = torch.randn(200, 4, 64).bfloat16().cuda()

    def call(cu, max_q=150, lens=(150, 60), tables=None):
        out, lse = torch.full_like(q, 3.0), torch.full((200, 4), 5.0, device="cuda")
        B.pa_prefill_window(q, torch.tensor(cu, dtype=torch.int32).cuda(), b.kc, b.vc,
                            (b.tables if tables is None else tables).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                            0.125, out, max_q, 150, lse=lse)
        return out, lse, B.pa_get_device_error()[0]
    out, lse, st = call([1, 131, 190])
    assert st == B.PA_OK
    s = slice(1, 131)
    _check_rows(q[s].cpu(), out[s].cpu(), lse[s].cpu(), b.rows[0][0], b.rows[1][0], 0, 0.0, None)
    for x, v in ((out, 3.0), (lse, 5.0)):
        assert (x[:1] == v).all() and (x[190:] == v).all()
    for cu, max_q in (([1, 140, 190], 130), ([0, 100, 201 - 50 + 100], 150), ([-1, 100, 150], 150), ([60, 50, 100], 150)):
        assert call(cu, max_q)[2] == B.PA_ERR_DEVICE_BOUNDS
    left = call([1, 140, 190], 130)[0]
    assert (left[:140] == 3.0).all() and torch.equal(left[140:190], call([1, 140, 190])[0][140:190])
    assert call([1, 131, 190], lens=(151, 60))[2] == B.PA_ERR_DEVICE_BOUNDS
    for bad in (-1, b.kc.shape[0], 2 ** 31 - 1):
        tables = b.tables.clone()
        tables[0, 1] = bad
        again, _, st = call([1, 131, 190], tables=tables)
        assert st == B.PA_ERR_DEVICE_BOUNDS and torch.equal(again[131:190], out[131:190])


def test_captured_repeated_and_on_another_stream():
    b = Batch([700, 300], 2, 128, 16, "bf16", seed=3)
    counts = [600, 130]
    q = torch.randn(730, 8, 128, generator=b.g).bfloat16().cuda()
    cu, tables = torch.tensor([0, 600, 730], dtype=torch.int32).cuda(), b.tables.cuda()
    lens = torch.tensor([700, 300], dtype=torch.int32).cuda()

    def call(out):
        B.pa_prefill_window(q, cu, b.kc, b.vc, tables, lens, 128 ** -0.5, out, 600, 700, window=150)
    first, again, out_g, out_s = (torch.empty_like(q) for _ in range(4))
    call(first)
    call(again)
    assert torch.equal(first, again)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(out_g)
    graph.replay()
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.default_stream())
        call(out_s)
    torch.cuda.synchronize()
    assert torch.equal(first, out_g) and torch.equal(first, out_s)
    lens.copy_(torch.tensor([650, 131], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    b.rows = [[x[:n] for x, n in zip(rows, (650, 131))] for rows in b.rows]
    _check(b, counts, q.cpu(), out_g.cpu(), None, 150)


def test_wrong_tensors_are_refused():
    b = Batch([50, 60], 2, 64, 16, "bf16")
    q = torch.randn(40, 4, 64).bfloat16().cuda()
    cu = torch.tensor([0, 20, 40], dtype=torch.int32).cuda()
    args = dict(q=q, cu_q_lens=cu, k_cache=b.kc, v_cache=b.vc, block_tables=b.tables.cuda(),
                context_lens=torch.tensor([50, 60], dtype=torch.int32).cuda(), scale=0.125, out=torch.empty_like(q),
                max_q_len=20, max_context_len=60)
    B.pa_prefill_window(**args)
    for kw in (dict(q=q.float()), dict(out=torch.empty(40, 4, 64, device="cuda")), dict(cu_q_lens=None),
               dict(cu_q_lens=cu[:2]), dict(block_tables=b.tables.cuda()[:1]), dict(sinks=torch.zeros(3, device="cuda")),
               dict(lse=torch.zeros(40, 3, device="cuda")), dict(q=q[:, :, :32])):
        with pytest.raises((TypeError, ValueError)):
            B.pa_prefill_window(**dict(args, **kw))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_a_layer_as_it_is_served(dtype):
    """Prompts, single steps and drafts of one layer with rotary positions, a
    window and sinks, by the cache's own calls, against the oracle over the whole
    history: rows rotated in fp32 and stored as the cache stores them."""
    from oracle import fp8
    hq, hkv, D, window = 8, 2, 64, 40
    ks, vs = 0.011, 0.017
    g = torch.Generator().manual_seed(12)
    cache = PagedKVCache(60, hkv, 16, D, {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}[dtype], "cuda",
                         fill=float("nan"), k_scale=ks, v_scale=vs)
    table, sinks = B.rotary_table(400, D), _sinks(hq)
    cs = table.cpu().numpy()
    hist = {s: ([], []) for s in (0, 1, 2)}

    def stored(x32, scale):
        if dtype == "bf16":
            return torch.from_numpy(np.ascontiguousarray(x32)).bfloat16().double().numpy()
        return fp8.dequantize(fp8.quantize(x32, scale), scale)
    for ids, counts in (([0, 1], [150, 33]), ([1, 0], [1, 1]), ([0, 1, 2], [4, 1, 20]), ([2, 0, 1], [5, 1, 3]),
                        ([0, 2], [1, 1]), ([1, 2], [60, 1])):
        T = sum(counts)
        qkv = torch.randn(T, (hq + 2 * hkv) * D, generator=g).bfloat16()
        q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.cuda().split([hq * D, hkv * D, hkv * D], 1))
        pos = np.concatenate([np.arange(len(hist[s][0]), len(hist[s][0]) + c) for s, c in zip(ids, counts)])
        q_rot = cache.append_rotated(ids, counts, q, k, v, table)
        lse = torch.empty(T, hq, device="cuda")
        out = cache.attend(ids, counts, q_rot, window=window, sinks=sinks.cuda(), lse=lse)
        x = qkv.float().numpy().reshape(T, -1, D)
        turned = rotate(x[:, :hq + hkv], cs[pos, :D // 2], cs[pos, D // 2:], False)
        qr = torch.from_numpy(turned[:, :hq]).bfloat16()
        assert torch.equal(q_rot.cpu(), qr)
        at = 0
        for s, c in zip(ids, counts):
            hist[s][0].extend(stored(turned[at:at + c, hq:], ks))
            hist[s][1].extend(stored(np.ascontiguousarray(x[at:at + c, hq + hkv:]), vs))
            _check_rows(qr[at:at + c], out[at:at + c].cpu(), lse[at:at + c].cpu(), np.stack(hist[s][0]),
                        np.stack(hist[s][1]), window, 0.0, sinks.double().numpy())
            at += c
    assert B.pa_get_device_error()[0] == B.PA_OK


def test_cache_calls_are_all_or_nothing():
    cache = PagedKVCache(4, 2, 16, 64, torch.bfloat16, "cuda")
    table = B.rotary_table(200, 64)
    rows = lambda n, h=2: torch.randn(n, h, 64).bfloat16().cuda()
    cache.append_rotated([0], [30], rows(30, 4), rows(30), rows(30), table)
    before = (dict(cache.lens), cache.bm.stats())
    for ids, counts in (([0, 5], [3, 40]), ([5, 0], [16, 30]), ([0, 0], [1, 1]), ([0], [-1]), ([0, 5], [3])):
        T = max(0, sum(counts))
        with pytest.raises((B.PagedAttnError, ValueError)):
            cache.append_rotated(ids, counts, rows(T, 4), rows(T), rows(T), table)
        assert (dict(cache.lens), cache.bm.stats()) == before
    good = [rows(2, 4), rows(2), rows(2), table]
    for i, bad in ((0, good[0].float()), (1, rows(2, 3)), (2, rows(3)), (2, good[2].cpu()), (3, table.double()),
                   (3, table[:, :24].contiguous()), (3, table[:, :8].contiguous()), (0, rows(2, 0)),
                   (1, torch.randn(2, 133).bfloat16().cuda()[:, 1:129].view(2, 2, 64)),
                   (0, torch.randn(2 * 256 + 1).bfloat16().cuda()[1:].view(2, 4, 64))):
        with pytest.raises((B.PagedAttnError, ValueError, TypeError)):
            cache.append_rotated([0], [2], *[bad if i == k else x for k, x in enumerate(good)])
        assert (dict(cache.lens), cache.bm.stats()) == before
    with pytest.raises(ValueError):
        cache.append_rotated([0], [2], rows(3, 4), rows(3), rows(3), table)
    with pytest.raises(ValueError):
        cache.append_rotated([0], [9], rows(9, 4), rows(9), rows(9), table[:38])
    with pytest.raises(ValueError):
        cache.attend([0], [31], rows(31, 4))
    assert cache.attend([], [], rows(0, 4)).shape == (0, 4, 64)
