"""pa_decode_multi against the oracle in 64 bits.

Bounds, for |q|, |k|, |v| of N(0, 1) and scale D^-1/2. A score is a sum of D
products in fp32, off by at most D 2^-24 sum|q_i k_i| scale < 1e-4 (D 128: the
sum is near 82, the scale 0.088); a capped one by a few 2^-24 of twice the cap
in base 2 more (cap 50: 2e-5). So a weight over the denominator is off by 2e-4
of itself at most, and by its rounding: with up to 8 rows (new tokens x query
heads of a kv head) over a bf16 cache it is split in two bf16 (2^-16), otherwise
rounded to f16 (half a step, 2^-11). With size = sum_j w_j |v_j| / den, the
result before its rounding to bf16 (half a step, 2^-8 of itself) is off by at
most W size, W = 2^-12 where it is split, else 2^-11 + 2^-12: for a weight
w' = w (1 + e), |e| <= 2^-11, |sum w'_j v_j - sum w_j v_j| / den <= 2^-11 size,
and the denominator sums the weights before that rounding. With more than 8
rows V too is f16: exact from 2^-14 up, off by 2^-25 at most below, which a
weighted mean does not enlarge (2^-24 for the bound, over bf16).
The log-sum-exp is off by the score's error, at most 1.2e-4 with the base
changes, and its own rounding.
"""
import numpy as np
import pytest
import torch

from oracle import fp8, int8
from oracle.options import options_attention
from paged_kv_cache_361_b200 import binding as B

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}
SCALE = {"bf16": (1.0, 1.0), "e4m3": (0.011, 0.017), "int8": (0.031, 0.027)}
W = 2.0 ** -11 + 2.0 ** -12
W_SPLIT = 2.0 ** -12
LSE = 1.2e-4


@pytest.fixture(autouse=True)
def _clean_error_word():
    B.pa_get_device_error()
    yield


class Batch:
    """A paged cache filled with N(0, 1) rows and its logical rows in fp64.
    Blocks of no sequence, and the slots behind a sequence's last token, hold
    NaN (int8: the code -128)."""

    def __init__(self, lens, hkv, D, bs, dtype, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.bs, self.dtype, self.lens = bs, dtype, list(lens)
        blocks = [-(-x // bs) for x in lens]
        nb = sum(blocks) + 2
        order = torch.randperm(nb, generator=g)
        self.max_blocks = max(1, max(blocks))
        self.tables = torch.full((len(lens), self.max_blocks), -1, dtype=torch.int32)
        pools, self.rows = [], []
        at = 0
        for i, b in enumerate(blocks):
            self.tables[i, :b] = order[at:at + b].int()
            at += b
        for which in (0, 1):
            sc = SCALE[dtype][which]
            pool = torch.zeros(nb, hkv, bs, D, dtype=DT[dtype])
            pool.view(torch.uint8).fill_({"bf16": 0xFF, "e4m3": 0x7F, "int8": 0x80}[dtype])
            logical = []
            for i, x in enumerate(lens):
                rows = torch.randn(x, hkv, D, generator=g)
                if dtype == "bf16":
                    stored = rows.bfloat16()
                    value = stored.double().numpy()
                else:
                    q = fp8 if dtype == "e4m3" else int8
                    codes = q.quantize(rows.numpy(), sc)
                    stored = torch.from_numpy(codes).view(DT[dtype])
                    value = q.dequantize(codes, sc)
                t = torch.arange(x)
                ids = self.tables[i].long()[t // bs]
                flat = pool.view(torch.uint8) if dtype != "bf16" else pool.view(torch.int16)
                flat[ids, :, t % bs] = stored.view(flat.dtype)
                logical.append(value)
            pools.append(pool.cuda())
            self.rows.append(logical)
        self.kc, self.vc = pools
        if dtype != "bf16":
            B.set_kv_scales(self.kc, self.vc, *SCALE[dtype])
        self.g = g

    def run(self, counts, hq, window=0, cap=0.0, sinks=None, P=-1, tables=None, want_lse=True, cu=True, max_ctx=None,
            max_q=None):
        T, D = sum(counts), self.kc.shape[3]
        q = torch.randn(T, hq, D, generator=self.g).bfloat16()
        out = torch.full((T, hq, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        lse = torch.full((T, hq), float("nan"), device="cuda") if want_lse else None
        max_ctx = max(self.lens) if max_ctx is None else max_ctx
        max_q = max(counts) if max_q is None else max_q
        need = B.pa_decode_multi_workspace_bytes(T, len(counts), max_q, hq, self.kc.shape[1], D, max_ctx, window, P)
        ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")
        cu_t = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32).cuda() if cu else None
        B.pa_decode_multi(q.cuda(), cu_t, self.kc, self.vc, (self.tables if tables is None else tables).cuda(),
                          torch.tensor(self.lens, dtype=torch.int32).cuda(), D ** -0.5, out, max_q, max_ctx,
                          window=window, softcap=cap, sinks=None if sinks is None else sinks.cuda(), lse=lse,
                          partition_tokens=P, workspace=ws)
        torch.cuda.synchronize()
        return q, out.cpu(), None if lse is None else lse.cpu()

    def check(self, counts, q, out, lse, window=0, cap=0.0, sinks=None):
        hq, hkv = q.shape[1], self.kc.shape[1]
        f16 = self.dtype != "bf16" or max(counts) * (hq // hkv) > 8
        at = 0
        for i, n in enumerate(counts):
            ref, want, size = options_attention(q[at:at + n], self.rows[0][i], self.rows[1][i], q.shape[2] ** -0.5,
                                                window, cap, None if sinks is None else sinks.double().numpy())
            got = out[at:at + n].double().numpy()
            tol = 2.0 ** -8 * np.abs(ref) + (W if f16 else W_SPLIT) * (1 + 2.0 ** -8) * size + (2.0 ** -24 if f16 else 0)
            assert (np.abs(got - ref) <= tol).all(), (i, float((np.abs(got - ref) - tol).max()))
            if lse is not None:
                gl = lse[at:at + n].double().numpy()
                fin = np.isfinite(want)
                assert np.array_equal(gl[~fin], want[~fin])
                assert (np.abs(gl - want)[fin] <= LSE + 2.0 ** -23 * np.abs(want[fin])).all()
            at += n


def _sinks(hq, seed=1):
    return torch.randn(hq, generator=torch.Generator().manual_seed(seed))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("bs", [8, 16, 32])
def test_shapes(dtype, D, G, bs):
    """Lengths around blocks and chunks, from one row to 128 (both kernels, every
    number of softmax warps), split and not."""
    lens = [1, 7, 63, 64, 65, 130, 391]
    b = Batch(lens, 2, D, bs, dtype, seed=D + G + bs)
    for counts, window, cap, sink, P in (
            ([1] * 7, 0, 0.0, False, -1), ([1, 3, 2, 0, 4, 1, 5], 0, 0.0, True, 64), ([1, 7, 16, 1, 9, 16, 13], 50, 0.0, True, 128),
            ([1, 2, 1, 2, 1, 2, 2], 17, 30.0, False, 0), ([1, 5, 4, 3, 2, 1, 6], 64, 50.0, True, 64)):
        sinks = _sinks(2 * G) if sink else None
        b.check(counts, *b.run(counts, 2 * G, window, cap, sinks, P), window, cap, sinks)
    assert B.pa_get_device_error()[0] == B.PA_OK


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("window", [1, 2, 15, 16, 64, 65, 200, 391, 392, 10 ** 6])
def test_windows(dtype, window):
    """Windows of one key, around chunks, of the context and past it; drafts
    longer than the window; blocks wholly before every window are gone: their
    table entries are -1 and their bytes NaN."""
    lens = [391, 64, 5, 200]
    b = Batch(lens, 2, 64, 16, dtype, seed=window % 97)
    for counts in ([1, 1, 1, 1], [16, 3, 5, 7]):
        tables = b.tables.clone()
        for i, (L, n) in enumerate(zip(lens, counts)):
            first = max(0, L - n - window + 1)
            for e in range(first // 16):
                b.kc.view(torch.uint8)[tables[i, e]] = 0xFF if dtype == "bf16" else 0x7F
                b.vc.view(torch.uint8)[tables[i, e]] = 0xFF if dtype == "bf16" else 0x7F
                tables[i, e] = -1
        for P in (0, 64, -1):
            b.check(counts, *b.run(counts, 8, window, 0.0, None, P, tables=tables), window)
        assert B.pa_get_device_error()[0] == B.PA_OK
        b = Batch(lens, 2, 64, 16, dtype, seed=window % 97 + 1)


def test_sinks_of_every_size():
    """No weight (-inf), far above and far below the scores."""
    b = Batch([40, 1, 300], 2, 128, 16, "bf16")
    sinks = torch.tensor([float("-inf"), 1e4, -1e4, 0.0, 80.0, -80.0, 3.0, float("-inf")])
    for counts in ([1, 1, 1], [5, 1, 3]):
        for P in (0, 64):
            b.check(counts, *b.run(counts, 8, 0, 0.0, sinks, P), 0, 0.0, sinks)


def test_empty_contexts_and_one_row_per_sequence():
    """cu_q_lens NULL: a sequence of length 0 gets a zero row and its sink."""
    b = Batch([5, 0, 70], 2, 64, 8, "bf16")
    for sinks in (None, _sinks(4)):
        for P in (0, 64):
            q, out, lse = b.run([1, 1, 1], 4, 3, 0.0, sinks, P, cu=False)
            b.check([1, 1, 1], q, out, lse, 3, 0.0, sinks)
            assert not out[1].any()
    assert B.pa_get_device_error()[0] == B.PA_OK
    b = Batch([0, 0], 2, 64, 8, "bf16")
    q, out, lse = b.run([1, 1], 4, cu=False)
    assert not out.any() and (lse == float("-inf")).all()


def test_many_empty_and_short_sequences_between_long_ones():
    """Runs of sequences without rows, without keys (more tokens than context is an
    error; so is none) and of one key, between ones that several CTAs share."""
    lens = [0, 3000, 1, 1, 0, 0, 1, 0, 2500, 1, 1, 1, 64, 0, 1, 700, 0]
    for G in (1, 2, 8):
        b = Batch(lens, 2, 64, 16, "bf16", seed=G)
        for P in (-1, 0, 64, 448):
            counts = [1] * len(lens)
            b.check(counts, *b.run(counts, 2 * G, 0, 0.0, _sinks(2 * G), P, cu=False), 0, 0.0, _sinks(2 * G))
            counts = [min(x, (i * 5) % 7) for i, x in enumerate(lens)]
            b.check(counts, *b.run(counts, 2 * G, 900, 0.0, None, P), 900)
    assert B.pa_get_device_error()[0] == B.PA_OK


def test_even_shares_over_a_large_ragged_batch():
    """300 sequences from 1 to 1900 tokens, so that every CTA has several segments."""
    g = torch.Generator().manual_seed(77)
    lens = torch.randint(1, 1900, (300,), generator=g).tolist()
    counts = [min(x, int(n)) for x, n in zip(lens, torch.randint(0, 5, (300,), generator=g))]
    for dtype, G in (("bf16", 2), ("int8", 1), ("bf16", 8), ("e4m3", 4)):
        b = Batch(lens, 1, 64, 16, dtype, seed=G)
        for window in (0, 300):
            b.check(counts, *b.run(counts, G, window), window)
            b.check([1] * 300, *b.run([1] * 300, G, window, cu=False), window)
    assert B.pa_get_device_error()[0] == B.PA_OK


@pytest.mark.parametrize("num,hkv,n,window", [(5000, 1, 1, 0), (5000, 2, 3, 40), (700, 8, 16, 0)])
def test_more_sequences_than_threads(num, hkv, n, window):
    """Far more units than CTAs, by even shares, by shares of 256 keys and a unit at a
    time. Two results are each W size (size up to the largest |v|) off before their
    rounding, and half a step of bf16; two log-sum-exps LSE and a rounding."""
    g = torch.Generator().manual_seed(num)
    L = torch.randint(n, 301, (num,), generator=g, dtype=torch.int32)
    blocks = (L + 15) // 16
    at = torch.cumsum(blocks, 0) - blocks
    tables = (at[:, None] + torch.arange(19)).int()       # entries past a sequence's blocks are not used
    nb = int(blocks.sum())
    tables[tables >= nb] = -1
    kc, vc = (torch.randn(nb, hkv, 16, 64, generator=g).bfloat16().cuda() for _ in range(2))
    q = torch.randn(num * n, 4 * hkv, 64, generator=g).bfloat16().cuda()
    cu = (torch.arange(num + 1, dtype=torch.int32) * n).cuda()
    got = []
    for P in (-1, 0, 256):
        out, lse = torch.full_like(q, float("nan")), torch.full(q.shape[:2], float("nan"), device="cuda")
        need = B.pa_decode_multi_workspace_bytes(num * n, num, n, 4 * hkv, hkv, 64, 300, window, P)
        B.pa_decode_multi(q, cu, kc, vc, tables.cuda(), L.cuda(), 0.125, out, n, 300, window=window, lse=lse,
                          partition_tokens=P, workspace=torch.full((need,), 255, dtype=torch.uint8, device="cuda"))
        got.append((out.double(), lse.double()))
    assert B.pa_get_device_error()[0] == B.PA_OK
    top = float(vc.abs().max())
    for out, lse in got[::2]:
        assert ((out - got[1][0]).abs() <= 2.0 ** -8 * (out.abs() + got[1][0].abs()) + 2 * W * top).all()
        assert ((lse - got[1][1]).abs() <= 2 * LSE + 2.0 ** -23 * lse.abs()).all()


def test_partitions_agree_and_long_context():
    b = Batch([9000, 4097, 1, 6500], 2, 128, 32, "bf16", seed=5)
    for counts, window in (([1, 1, 1, 1], 0), ([4, 2, 1, 3], 5000), ([4, 4, 1, 16], 0)):
        for P in (-1, 64, 1024, 0):
            b.check(counts, *b.run(counts, 16, window, 0.0, None, P), window)


def test_scores_that_grow_along_the_sequence():
    """Every key of the second half outweighs those before it by far (the running
    maximum moves), and the capped form saturates."""
    b = Batch([257, 640], 1, 64, 16, "bf16", seed=9)
    D = 64
    q = torch.ones(2, 4, D).bfloat16()
    for i, L in enumerate(b.lens):
        ramp = torch.linspace(-6, 6, L)[:, None, None].expand(L, 1, D).bfloat16()
        t = torch.arange(L)
        b.kc[b.tables[i].long()[t // 16].cuda(), :, (t % 16).cuda()] = ramp.cuda()
        b.rows[0][i] = ramp.double().numpy()
    for cap in (0.0, 20.0):
        for P in (0, 128):
            out = torch.empty(2, 4, D, dtype=torch.bfloat16, device="cuda")
            lse = torch.empty(2, 4, device="cuda")
            ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
            B.pa_decode_multi(q.cuda(), None, b.kc, b.vc, b.tables.cuda(), torch.tensor(b.lens, dtype=torch.int32).cuda(),
                              D ** -0.5, out, 1, 640, softcap=cap, lse=lse, partition_tokens=P, workspace=ws)
            b.check([1, 1], q, out.cpu(), lse.cpu(), 0, cap)


def test_rows_of_no_sequence_stay():
    b = Batch([50, 60], 2, 64, 16, "bf16")
    q = torch.randn(9, 4, 64).bfloat16().cuda()
    for P in (0, 64):
        out, lse = torch.full_like(q, 3.0), torch.full((9, 4), 5.0, device="cuda")
        ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
        cu = torch.tensor([1, 3, 6], dtype=torch.int32).cuda()     # rows 0, 6, 7, 8 belong to nobody
        B.pa_decode_multi(q, cu, b.kc, b.vc, b.tables.cuda(), torch.tensor([50, 60], dtype=torch.int32).cuda(), 0.125,
                          out, 3, 60, lse=lse, partition_tokens=P, workspace=ws)
        b.check([2, 3], q[1:6].cpu(), out[1:6].cpu(), lse[1:6].cpu())
        for x, v in ((out, 3.0), (lse, 5.0)):
            assert (x[[0, 6, 7, 8]] == v).all()


def test_bad_lengths_rows_and_blocks_are_recorded():
    """Each is recorded, and the sequences that are in order are computed."""
    b = Batch([50, 60], 2, 64, 16, "bf16")
    q = torch.randn(4, 4, 64).bfloat16().cuda()
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")

    def call(cu, lens, tables=None, max_q=2):
        out, lse = torch.full_like(q, 3.0), torch.full((4, 4), 5.0, device="cuda")
        B.pa_decode_multi(q, torch.tensor(cu, dtype=torch.int32).cuda(), b.kc, b.vc,
                          (b.tables if tables is None else tables).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                          0.125, out, max_q, 60, lse=lse, partition_tokens=64, workspace=ws)
        return out, lse, B.pa_get_device_error()[0]
    good = call([0, 2, 4], [50, 60])
    assert good[2] == B.PA_OK
    for cu, lens in (([0, 2, 4], [61, 60]), ([0, 2, 4], [-5, 60]), ([0, 2, 4], [1, 60])):
        out, _, st = call(cu, lens)
        assert st == B.PA_ERR_DEVICE_BOUNDS and torch.equal(out[2:], good[0][2:])
    for cu in ([0, 3, 4], [0, -1, 4], [2, 2, 5], [0, 2, 2 ** 31 - 1], [-7, 0, 2], [5, 6, 7]):
        assert call(cu, [50, 60])[2] == B.PA_ERR_DEVICE_BOUNDS
    for bad in (-1, b.kc.shape[0], 2 ** 31 - 1):
        tables = b.tables.clone()
        tables[0, 1] = bad
        out, _, st = call([0, 2, 4], [50, 60], tables)
        assert st == B.PA_ERR_DEVICE_BOUNDS and torch.equal(out[2:], good[0][2:])


def test_same_bits_every_time_and_in_a_graph():
    """No atomics: repeated calls agree bit for bit, and so do a captured and
    replayed call (with new lengths in the same buffers) and one on another stream."""
    lens = [3000, 1700, 64, 1]
    b = Batch(lens, 2, 128, 16, "bf16", seed=3)
    counts = [4, 1, 3, 1]
    T, hq = sum(counts), 8
    q = torch.randn(T, hq, 128, generator=b.g).bfloat16().cuda()
    cu = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32).cuda()
    tables, lens_d = b.tables.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    need = B.pa_decode_multi_workspace_bytes(T, 4, 4, hq, 2, 128, 3000, 2500, 256)
    assert need

    def call(out, ws):
        B.pa_decode_multi(q, cu, b.kc, b.vc, tables, lens_d, 128 ** -0.5, out, 4, 3000, window=2500,
                          partition_tokens=256, workspace=ws)
    first = torch.empty_like(q)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    call(first, ws)
    for _ in range(3):
        again = torch.empty_like(q)
        call(again, ws)
        assert torch.equal(first, again)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out_g, ws_g = torch.zeros_like(q), torch.empty(need, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(out_g, ws_g)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, out_g)
    with torch.cuda.stream(side):                 # another stream, its own workspace, at the same time
        out_s, ws_s = torch.zeros_like(q), torch.empty(need, dtype=torch.uint8, device="cuda")
        side.wait_stream(torch.cuda.default_stream())
        call(out_s, ws_s)
    call(again, ws)
    torch.cuda.synchronize()
    assert torch.equal(first, out_s) and torch.equal(first, again)
    lens_d.copy_(torch.tensor([2000, 900, 64, 1], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    b.lens = [2000, 900, 64, 1]
    b.rows = [[x[:n] for x, n in zip(rows, b.lens)] for rows in b.rows]
    b.check(counts, q.cpu(), out_g.cpu(), None, 2500)


def test_wrong_tensors_are_refused():
    b = Batch([50, 60], 2, 64, 16, "bf16")
    q = torch.randn(4, 4, 64).bfloat16().cuda()
    cu = torch.tensor([0, 2, 4], dtype=torch.int32).cuda()
    args = dict(q=q, cu_q_lens=cu, k_cache=b.kc, v_cache=b.vc, block_tables=b.tables.cuda(),
                context_lens=torch.tensor([50, 60], dtype=torch.int32).cuda(), scale=0.125, out=torch.empty_like(q),
                max_q_len=2, max_context_len=60, partition_tokens=0)
    B.pa_decode_multi(**args)
    for kw in (dict(q=q.float()), dict(out=torch.empty(4, 4, 64, device="cuda")), dict(cu_q_lens=cu[:2]),
               dict(cu_q_lens=cu.long()), dict(block_tables=b.tables.cuda()[:1]), dict(context_lens=args["context_lens"].cpu()),
               dict(sinks=torch.zeros(3, device="cuda")), dict(sinks=torch.zeros(4).cuda().double()),
               dict(lse=torch.zeros(4, 3, device="cuda")), dict(q=q[:, :, :32]), dict(lse=torch.zeros(4, 4))):
        with pytest.raises((TypeError, ValueError)):
            B.pa_decode_multi(**dict(args, **kw))
    for kw, st in ((dict(max_q_len=17), B.PA_ERR_UNSUPPORTED),
                   (dict(partition_tokens=64, max_context_len=128, block_tables=torch.zeros(2, 8, dtype=torch.int32).cuda()),
                    B.PA_ERR_INVALID_ARG),  # two chunks a unit: a workspace is needed
                   (dict(window=-1), B.PA_ERR_INVALID_ARG)):
        with pytest.raises(B.PagedAttnError) as e:
            B.pa_decode_multi(**dict(args, **kw))
        assert e.value.status == st
