"""Cases of the serving operators for rotary, windowed and multi-token attention over the paged KV cache.

Three operators, as a serving loop runs them layer by layer:
  rotate   pa_rotate_and_cache: rotate q and k by their positions, append k and v to the cache
  multi    pa_decode_multi: attention of one or a few new tokens per sequence, split over the cache's length
  window   pa_prefill_window: causal attention of whole prompts or prompt chunks
multi and window take a sliding window, a score cap and per-head sinks, and return the log-sum-exp of every row.

`run` computes them in plain torch, or with `own` by the calls a user makes.
"""
import math

import torch

own = False

DEV = "cuda"
CACHE_DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}
# powers of two: N(0, 1) values use most of the codes
SCALE = {"bf16": 1.0, "f32": 1.0, "e4m3": 2.0 ** -6, "int8": 2.0 ** -5}
ELEM = {"bf16": 2, "f32": 4, "e4m3": 1, "int8": 1}


def listed():
    return [
        # a decode step of 64 sequences, grouped heads: latency counts
        dict(name="rotate step", op="rotate", tokens=64, seqs=64, hq=32, hkv=8, d=128, bs=16, dtype="bf16", rd=128,
             pairs="half", pos=8192),
        # a small ragged batch over an int8 cache, neighbouring pairs
        dict(name="rotate step int8", op="rotate", tokens=7, seqs=7, hq=64, hkv=8, d=64, bs=32, dtype="int8", rd=64,
             pairs="next", pos=4096),
        # whole prompts, one kv head per query head
        dict(name="rotate prompts", op="rotate", tokens=16231, seqs=8, hq=32, hkv=32, d=128, bs=16, dtype="bf16",
             rd=128, pairs="half", pos=4096),
        # prompts into an 8-bit cache, half of each head rotated, far positions
        dict(name="rotate prompts e4m3", op="rotate", tokens=20011, seqs=4, hq=64, hkv=8, d=128, bs=32, dtype="e4m3",
             rd=64, pairs="half", pos=131072),
        # a windowed layer's decode step
        dict(name="window step", op="multi", seqs=64, n=1, n_lo=1, lo=128, hi=8192, hq=32, hkv=8, d=128, bs=16,
             dtype="bf16", window=1024, cap=0.0, sinks=True),
        # drafts of 5 tokens verified against long contexts
        dict(name="draft check", op="multi", seqs=16, n=5, n_lo=5, lo=1000, hi=32768, hq=64, hkv=8, d=128, bs=32,
             dtype="bf16", window=0, cap=0.0, sinks=False),
        # one sequence with a very long 8-bit cache
        dict(name="long step e4m3", op="multi", seqs=1, n=1, n_lo=1, lo=131072, hi=131072, hq=64, hkv=8, d=128, bs=32,
             dtype="e4m3", window=0, cap=50.0, sinks=False),
        # a mixed batch (some sequences one token, some four), one kv head per query head, int8
        dict(name="mixed step int8", op="multi", seqs=32, n=4, n_lo=1, lo=128, hi=2048, hq=32, hkv=32, d=128, bs=16,
             dtype="int8", window=0, cap=0.0, sinks=False),
        # a few sequences that have just begun: the smallest call
        dict(name="short step", op="multi", seqs=3, n=1, n_lo=1, lo=1, hi=40, hq=8, hkv=4, d=64, bs=8, dtype="bf16",
             window=0, cap=0.0, sinks=True),
        # two prompts through a windowed layer with sinks
        dict(name="window prompts", op="window", seqs=2, n=4096, n_lo=3001, pre=0, hq=64, hkv=8, d=128, bs=16,
             dtype="bf16", window=1024, cap=0.0, sinks=True),
        # eight prompts through a layer with capped scores
        dict(name="capped prompts", op="window", seqs=8, n=2048, n_lo=700, pre=0, hq=32, hkv=32, d=128, bs=16,
             dtype="bf16", window=0, cap=50.0, sinks=False),
        # ragged chunks behind what an 8-bit cache already holds
        dict(name="window chunks e4m3", op="window", seqs=6, n=512, n_lo=33, pre=8000, hq=32, hkv=8, d=64, bs=32,
             dtype="e4m3", window=700, cap=30.0, sinks=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotate", "multi", "window"])
    hkv = rng.choice([1, 2, 4, 8, 16, 32])
    g = rng.choice([1, 2, 4, 8] if hkv <= 8 else [1, 2])
    d = rng.choice([64, 128])
    if op == "rotate":
        dtype = rng.choice(["bf16", "bf16", "f32", "e4m3", "int8"])
        tokens = min(_log(rng, 1, 20000), 110_000_000 // ((g + 2) * hkv * d * (2 if dtype == "f32" else 1)))
        return dict(op=op, tokens=tokens, seqs=min(tokens, _log(rng, 1, 64)), hq=g * hkv, hkv=hkv, d=d,
                    bs=rng.choice([1, 4, 8, 16, 32]), dtype=dtype, rd=rng.choice([d, d, d // 2]),
                    pairs=rng.choice(["half", "next"]), pos=_log(rng, tokens + 1, 262144))
    dtype = rng.choice(["bf16", "bf16", "e4m3", "int8"])
    bs = rng.choice([8, 16, 32])
    cap = rng.choice([0.0, 0.0, 30.0, 50.0])
    sinks = rng.choice([True, False])
    window = rng.choice([0, _log(rng, 1, 4096)])
    if op == "multi":
        seqs = _log(rng, 1, 128)
        most = min(131072, 250_000_000 // (seqs * hkv * d))
        hi = _log(rng, 20, max(21, most))
        n = rng.choice([1, 1, rng.randint(2, 16)])
        return dict(op=op, seqs=seqs, n=n, n_lo=rng.randint(1, n), lo=_log(rng, n, max(n, hi)), hi=max(n, hi), hq=g * hkv,
                    hkv=hkv, d=d, bs=bs, dtype=dtype, window=window, cap=cap, sinks=sinks)
    seqs = _log(rng, 1, 8)
    n = _log(rng, 17, 4096)
    pre = rng.choice([0, _log(rng, 1, 8192)])
    # the plain form's score matrix, and the work, stay below the largest listed case's
    n = max(17, min(n, int(1_350_000_000 * 64 // (d * seqs * g * hkv * (n + (min(pre, window) if window else pre))))))
    return dict(op=op, seqs=seqs, n=n, n_lo=rng.randint(1, n), pre=pre, hq=g * hkv, hkv=hkv, d=d, bs=bs, dtype=dtype,
                window=window, cap=cap, sinks=sinks)


def _spread(lo, hi, n):
    """n whole numbers over [lo, hi], unordered, the last one hi."""
    return [lo + (hi - lo) * ((i * 619 + 331) % 1009) // 1008 for i in range(n - 1)] + [hi]


def _lengths(case):
    """(new tokens, context length with them) of every sequence."""
    n = _spread(case["n_lo"], case["n"], case["seqs"])
    if case["op"] == "window":
        pre = _spread(case["pre"] // 3, case["pre"], case["seqs"])
        return n, [p + c for p, c in zip(pre, n)]
    return n, [max(x, c) for x, c in zip(_spread(case["lo"], case["hi"], case["seqs"]), n)]


def _rotate_lengths(case):
    base = case["tokens"] // case["seqs"]
    return [base + (i < case["tokens"] % case["seqs"]) for i in range(case["seqs"])]


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device=DEV)


def _prepare_rotate(case, g):
    hq, hkv, d, bs, rd = (case[k] for k in ("hq", "hkv", "d", "bs", "rd"))
    counts, tokens = _rotate_lengths(case), case["tokens"]
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    # one projection's rows, q | k | v: the operator takes the three as views of it
    qkv = torch.randn(tokens, (hq + 2 * hkv) * d, generator=g, device=DEV).to(dt)
    blocks = [-(-c // bs) for c in counts]
    order = torch.randperm(sum(blocks) + 3, generator=g, device=DEV)[:sum(blocks)]
    n = _ints(counts, torch.int64)
    seq = torch.repeat_interleave(torch.arange(case["seqs"], device=DEV), n)
    i = torch.arange(tokens, device=DEV) - (n.cumsum(0) - n)[seq]
    b = _ints(blocks, torch.int64)
    slots = order[(b.cumsum(0) - b)[seq] + i // bs] * bs + i % bs
    first = torch.randint(0, case["pos"] - max(counts) + 1, (case["seqs"],), generator=g, device=DEV)
    angles = torch.outer(torch.arange(case["pos"], device=DEV, dtype=torch.float64),
                         10000.0 ** (-torch.arange(0, rd, 2, device=DEV, dtype=torch.float64) / rd))
    cache = torch.zeros(sum(blocks) + 3, hkv, bs, d, device=DEV).to(CACHE_DTYPE[case["dtype"]])
    return dict(q=qkv[:, :hq * d].unflatten(1, (hq, d)), k=qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d)),
                v=qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d)), positions=(first[seq] + i).int(), slots=slots,
                table=torch.cat([angles.cos(), angles.sin()], 1).float(), k_cache=cache, v_cache=cache.clone())


def _prepare_attention(case, g):
    hq, hkv, d, bs = (case[k] for k in ("hq", "hkv", "d", "bs"))
    n, lens = _lengths(case)
    blocks = [-(-x // bs) for x in lens]
    total = sum(blocks) + 3
    order = torch.randperm(total, generator=g, device=DEV)[:sum(blocks)].int()
    tables = torch.full((case["seqs"], max(blocks)), -1, dtype=torch.int32, device=DEV)
    tables[torch.arange(max(blocks), device=DEV) < _ints(blocks)[:, None]] = order
    cu = [0]
    for c in n:
        cu.append(cu[-1] + c)
    scale = SCALE[case["dtype"]]

    def pool():
        x = torch.randn(total, hkv, bs, d, generator=g, device=DEV)
        if case["dtype"] == "int8":
            x = (x / scale).round_().clamp_(-127, 127)
        elif case["dtype"] == "e4m3":
            x = (x / scale).clamp_(-448, 448)
        return x.to(CACHE_DTYPE[case["dtype"]])

    # the first key that any row of a sequence sees
    first = [max(0, x - c - case["window"] + 1) if case["window"] else 0 for x, c in zip(lens, n)]
    return dict(q=torch.randn(cu[-1], hq, d, generator=g, device=DEV).bfloat16(), k_cache=pool(), v_cache=pool(),
                tables=tables, lens=_ints(lens), cu=_ints(cu), max_q=max(n), max_len=max(lens),
                sinks=torch.randn(hq, generator=g, device=DEV) if case["sinks"] else None, first=_ints(first),
                span=max(x - f for x, f in zip(lens, first)))


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return dict(_prepare_rotate(case, g) if case["op"] == "rotate" else _prepare_attention(case, g), case=case)


def _rotated(x, cos, sin, half):
    """x [T][H][D] with the first 2 * cos.shape[-1] dims of every head rotated, in 32 bits."""
    x, r = x.float(), 2 * cos.shape[-1]
    a, b = (x[..., :r // 2], x[..., r // 2:r]) if half else (x[..., 0:r:2], x[..., 1:r:2])
    y = (a * cos - b * sin, b * cos + a * sin)
    return torch.cat([torch.cat(y, -1) if half else torch.stack(y, -1).flatten(-2), x[..., r:]], -1)


def _to_cache(x, dtype, scale):
    if dtype == torch.int8:
        return (x / scale).round().clamp(-127, 127).to(dtype)
    if dtype == torch.float8_e4m3fn:
        return (x / scale).clamp(-448, 448).to(dtype)
    return x.to(dtype)


def _plain_rotate(s, case):
    cs = s["table"][s["positions"].long()][:, None]
    cos, sin = cs[..., :case["rd"] // 2], cs[..., case["rd"] // 2:]
    half, scale, dtype = case["pairs"] == "half", SCALE[case["dtype"]], s["k_cache"].dtype
    at, off = s["slots"] // case["bs"], s["slots"] % case["bs"]
    s["k_cache"][at, :, off] = _to_cache(_rotated(s["k"], cos, sin, half), dtype, scale)
    s["v_cache"][at, :, off] = _to_cache(s["v"].float(), dtype, scale)
    return _rotated(s["q"], cos, sin, half).to(s["q"].dtype)


def _plain_attention(s, case):
    hq, hkv, d, bs, window = (case[k] for k in ("hq", "hkv", "d", "bs", "window"))
    b, n, g = case["seqs"], s["max_q"], hq // hkv
    cu, lens = s["cu"].long(), s["lens"].long()
    count = cu[1:] - cu[:-1]
    # the visible keys of every sequence, gathered through its table
    key = s["first"].long()[:, None] + torch.arange(s["span"], device=DEV)
    inside = key < lens[:, None]
    key = torch.where(inside, key, 0)
    at, off = s["tables"].gather(1, key // bs).long(), key % bs
    scale = SCALE[case["dtype"]]
    keys = (s["k_cache"][at, :, off].float() * scale).transpose(1, 2)
    values = (s["v_cache"][at, :, off].float() * scale).transpose(1, 2)
    # the new tokens of every sequence, padded to the longest
    i = torch.arange(n, device=DEV)
    row = torch.where(i < count[:, None], cu[:-1, None] + i, 0)
    pos = (lens - count)[:, None] + i
    q = s["q"][row].float().view(b, n, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, g * n, d)
    x = torch.matmul(q, keys.transpose(2, 3)).mul_(d ** -0.5)
    if case["cap"]:
        x = x.div_(case["cap"]).tanh_().mul_(case["cap"])
    seen = inside[:, None] & (key[:, None] <= pos[..., None])
    if window:
        seen &= key[:, None] > pos[..., None] - window
    x = x.view(b, hkv, g, n, -1).masked_fill_(~seen[:, None, None], float("-inf"))
    top = x.amax(-1, keepdim=True)
    sink = None
    if s["sinks"] is not None:
        sink = s["sinks"].view(1, hkv, g, 1, 1)
        top = torch.maximum(top, sink)
    top = torch.where(top == float("-inf"), 0.0, top)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    if sink is not None:
        total = total + (sink - top).exp()
    out = torch.matmul(x.view(b, hkv, g * n, -1), values).view(b, hkv, g, n, d) / total
    lse = (top + total.log()).squeeze(-1)
    # back to the packed rows
    t = torch.arange(s["q"].shape[0], device=DEV)
    seq = torch.searchsorted(cu[1:], t, right=True)
    pick = (seq, t - cu[seq])
    return (out.permute(0, 3, 1, 2, 4).reshape(b, n, hq, d)[pick].to(torch.bfloat16),
            lse.permute(0, 3, 1, 2).reshape(b, n, hq)[pick])


def _own_rotate(s, case):
    from paged_kv_cache_361_b200 import binding as B
    if case["dtype"] in ("e4m3", "int8"):
        B.set_kv_scales(s["k_cache"], s["v_cache"], SCALE[case["dtype"]], SCALE[case["dtype"]])
    q_out = torch.empty(s["q"].shape, dtype=s["q"].dtype, device=DEV)
    B.pa_rotate_and_cache(s["q"], s["k"], s["v"], s["positions"], s["table"], s["slots"], s["k_cache"], s["v_cache"],
                          q_out, interleaved=case["pairs"] == "next")
    return q_out


def _own_attention(s, case):
    from paged_kv_cache_361_b200 import binding as B
    if case["dtype"] in ("e4m3", "int8"):
        B.set_kv_scales(s["k_cache"], s["v_cache"], SCALE[case["dtype"]], SCALE[case["dtype"]])
    q, hkv, d = s["q"], case["hkv"], case["d"]
    out = torch.empty(q.shape, dtype=q.dtype, device=DEV)
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device=DEV)
    rule = dict(window=case["window"], softcap=case["cap"], sinks=s["sinks"], lse=lse)
    if case["op"] == "multi":
        need = B.pa_decode_multi_workspace_bytes(q.shape[0], case["seqs"], s["max_q"], case["hq"], hkv, d, s["max_len"],
                                                 case["window"])
        B.pa_decode_multi(q, s["cu"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], d ** -0.5, out, s["max_q"],
                          s["max_len"], workspace=torch.empty(need, dtype=torch.uint8, device=DEV), **rule)
    else:
        B.pa_prefill_window(q, s["cu"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], d ** -0.5, out, s["max_q"],
                            s["max_len"], **rule)
    return out, lse


def run(state):
    case = state["case"]
    if case["op"] == "rotate":
        q = _own_rotate(state, case) if own else _plain_rotate(state, case)
        k, v = state["k_cache"], state["v_cache"]
        if case["dtype"] == "int8":  # the values that the codes stand for (exact in bf16: the scale is a power of two)
            k, v = (x.to(torch.bfloat16) * SCALE["int8"] for x in (k, v))
        return {"q": q, "k_cache": k, "v_cache": v}
    out, lse = _own_attention(state, case) if own else _plain_attention(state, case)
    return {"out": out, "lse": lse}


def work(case):
    hq, hkv, d, e = case["hq"], case["hkv"], case["d"], ELEM[case["dtype"]]
    if case["op"] == "rotate":
        t, x = case["tokens"], 4 if case["dtype"] == "f32" else 2
        return {"bytes": t * ((2 * hq + 2 * hkv) * d * x + 2 * hkv * d * e + 4 * case["rd"] + 12),
                "flops": 3 * t * (hq + hkv) * case["rd"]}
    n, lens = _lengths(case)
    w = case["window"]
    keys = sum(min(x, c + w - 1) if w else x for x, c in zip(lens, n))
    # pairs of a new token and a key that it sees: new token at position p sees min(p + 1, window) keys
    pairs = 0
    for x, c in zip(lens, n):
        lo, hi = x - c + 1, x  # visible counts without a window
        if w and lo >= w:
            pairs += c * w
        elif w and hi > w:
            pairs += (lo + w) * (w - lo + 1) // 2 + (hi - w) * w
        else:
            pairs += (lo + hi) * c // 2
    rows = sum(n) * hq
    return {"bytes": 2 * keys * hkv * d * e + rows * (4 * d + 4) + 4 * (-(-keys // case["bs"])) + 8 * case["seqs"],
            "flops": 4 * pairs * hq * d}


def _exact_rotate(s, case):
    rd, bs = case["rd"], case["bs"]
    pos = s["positions"].long()
    turn = torch.complex(s["table"][pos, :rd // 2].double(), s["table"][pos, rd // 2:].double())[:, None]

    def rotated(x):
        x = x.double().clone()
        if case["pairs"] == "half":
            z = torch.complex(x[..., :rd // 2], x[..., rd // 2:rd]) * turn
            x[..., :rd // 2], x[..., rd // 2:rd] = z.real, z.imag
        else:
            z = torch.complex(x[..., 0:rd:2], x[..., 1:rd:2]) * turn
            x[..., 0:rd:2], x[..., 1:rd:2] = z.real, z.imag
        return x

    def cached(x):
        pool = torch.zeros(s["k_cache"].shape, dtype=torch.float64, device=DEV).transpose(1, 2).reshape(-1, *x.shape[1:])
        scale = SCALE[case["dtype"]]
        if case["dtype"] == "int8":
            x = (x / scale).round().clamp(-127, 127) * scale
        elif case["dtype"] == "e4m3":  # steps of 2^(exponent - 3), the least exponent -6, codes without their scale
            x = (x / scale).clamp(-448, 448)
            step = torch.exp2(torch.frexp(x)[1].clamp(min=-5).double() - 4)
            x = (x / step).round() * step
        pool[s["slots"]] = x
        return pool.view(-1, bs, *x.shape[1:]).transpose(1, 2).contiguous()

    return {"q": rotated(s["q"]), "k_cache": cached(rotated(s["k"])), "v_cache": cached(s["v"].double())}


def _exact_attention(s, case):
    hq, hkv, d, bs, w = (case[k] for k in ("hq", "hkv", "d", "bs", "window"))
    g, scale = hq // hkv, SCALE[case["dtype"]]
    n, lens = _lengths(case)
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device=DEV)
    t0 = 0
    for i, (c, length) in enumerate(zip(n, lens)):
        ids = s["tables"][i, :-(-length // bs)].long()
        first = max(0, length - c - w + 1) if w else 0
        j = torch.arange(first, length, device=DEV)
        p = torch.arange(length - c, length, device=DEV)[:, None]
        hidden = (j > p) | (j <= p - w) if w else j > p
        for h in range(hkv):
            k, v = (x[ids, h].reshape(-1, d)[first:length].double() * scale for x in (s["k_cache"], s["v_cache"]))
            for u in range(h * g, h * g + g):
                z = s["q"][t0:t0 + c, u].double() @ k.T / math.sqrt(d)
                if case["cap"]:
                    z = case["cap"] * torch.tanh(z / case["cap"])
                z[hidden] = -math.inf
                norm = torch.logsumexp(z, 1)
                if s["sinks"] is not None:
                    norm = torch.logaddexp(norm, s["sinks"][u].double())
                out[t0:t0 + c, u] = torch.exp(z - norm[:, None]) @ v
                lse[t0:t0 + c, u] = norm
        t0 += c
    return {"out": out, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_rotate(s, case) if case["op"] == "rotate" else _exact_attention(s, case)
