"""The operators around the paged KV pool, as measured work.

Four operators that one serving step of a model runs in this order, each with a
plain form in elementary torch operations and a call of the framework's own
kernels (``own``):

* ``tables``   block tables and slot maps of a step, built on the GPU from the
               requests' lengths and a list of free pages;
* ``rope``     rotary positions (half or interleaved pairs, all or part of the
               head, any frequency scaling) of a step's q and k, with the
               append of k and v into the pool's pages;
* ``decode``, ``prefill``  attention over the paged cache whose scores are
               capped by a tanh, biased by distance, or limited to a window, a
               document or a prefix: one new token a sequence, or chunks;
* ``logprobs`` log-probabilities of given tokens with the entropy and the most
               likely alternatives.

Pool layout: bf16 [page][kv head][K, V][16 slots][64].
"""
import math

import torch

own = False

HEAD_DIM = 64
PAGE = 16
LOG2E = 1.4426950408889634


# ----------------------------------------------------------------------------
# the cases


def listed():
    return [
        # one decode step's bookkeeping of a 16-layer model: every request one token
        dict(name="tables_decode_64", op="tables", batch=64, layers=16, context=2048, prompts=0, chunk=0, capacity=64),
        # a mixed step of a 24-layer model: mostly decodes, some prompts, the token count padded
        dict(name="tables_mixed_256", op="tables", batch=256, layers=24, context=4096, prompts=12, chunk=1100, capacity=12000),
        # one decode step's rotation: pairs interleaved, half of the head rotated
        dict(name="rope_decode_64", op="rope", tokens=64, hq=14, hkv=2, rot=32, interleaved=True, context=4096, scaling="linear"),
        # a prompt batch at a long context: half pairs, the whole head, banded scaling
        dict(name="rope_prefill_8192", op="rope", tokens=8192, hq=32, hkv=8, rot=64, interleaved=False, context=32768, scaling="banded"),
        # a small decode batch of a model with capped scores: latency counts
        dict(name="decode_b8_cap", op="decode", batch=8, hq=32, hkv=8, lo=1, hi=2048, window=0, softcap=50.0, alibi=False, first=False, out="bf16"),
        # few long requests, distance bias, groups of seven heads
        dict(name="decode_b32_long_alibi", op="decode", batch=32, hq=14, hkv=2, lo=1000, hi=32768, window=0, softcap=0.0, alibi=True, first=False, out="bf16"),
        # a big batch on a local layer: capped scores over a window
        dict(name="decode_b256_cap_window", op="decode", batch=256, hq=32, hkv=8, lo=1, hi=8192, window=4096, softcap=50.0, alibi=False, first=True, out="bf16"),
        # prompts on a local layer with capped scores
        dict(name="prefill_4x2048_cap_window", op="prefill", batch=4, hq=32, hkv=8, chunk_lo=2048, chunk_hi=2048, start_hi=0, window=1024, softcap=50.0, alibi=False, doc=0, prefix=0, out="bf16"),
        # ragged chunks behind a cached part, packed documents, distance bias
        dict(name="prefill_ragged_docs_alibi", op="prefill", batch=7, hq=14, hkv=2, chunk_lo=1, chunk_hi=1500, start_hi=700, window=0, softcap=0.0, alibi=True, doc=400, prefix=0, out="bf16"),
        # one sampled token's scoring
        dict(name="logprobs_1", op="logprobs", rows=1, vocab=128256, top=20, dtype="bf16", scale=1.0, masked=False),
        # a decode batch's scoring, fp32 logits, temperature, some rows with few allowed tokens
        dict(name="logprobs_64_fp32", op="logprobs", rows=64, vocab=151936, top=5, dtype="fp32", scale=1.4, masked=True),
        # scoring a prompt
        dict(name="logprobs_2048", op="logprobs", rows=2048, vocab=128256, top=20, dtype="bf16", scale=1.0, masked=False),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["tables", "rope", "decode", "prefill", "logprobs"])
    hq, hkv = rng.choice([(32, 8), (14, 2), (8, 8), (16, 8), (15, 5), (20, 4), (12, 2), (16, 2)])
    softcap = rng.choice([0.0, 30.0, 50.0])
    window = rng.choice([0, spread(16, 4096)])
    out = rng.choice(["bf16", "bf16", "fp32"])
    if op == "tables":
        batch = spread(1, 256)
        prompts = rng.randint(0, min(batch, 12))
        chunk = spread(2, 1100)
        return dict(op=op, batch=batch, layers=rng.choice([1, 16, 24]), context=spread(32, 4096), prompts=prompts, chunk=chunk,
                    capacity=batch + prompts * chunk + rng.randint(0, 64))
    if op == "rope":
        return dict(op=op, tokens=spread(1, 8192), hq=hq, hkv=hkv, rot=8 * rng.randint(1, 8), interleaved=rng.random() < 0.5,
                    context=spread(64, 32768), scaling=rng.choice(["none", "linear", "banded"]))
    if op == "decode":
        batch = spread(1, 256)
        hi = min(spread(1, 32768), 2097152 // batch * 8 // hkv, 1048576 // batch)
        return dict(op=op, batch=batch, hq=hq, hkv=hkv, lo=rng.randint(1, hi), hi=hi, window=window, softcap=softcap,
                    alibi=rng.random() < 0.5, first=rng.random() < 0.3, out=out)
    if op == "prefill":
        batch = rng.randint(1, 8)
        start = rng.choice([0, spread(1, 1500)])
        n = spread(1, 2048)
        while batch * n * (n + start) * hq > 4 * 2048 * 2048 * 32:
            n = n * 3 // 4
        return dict(op=op, batch=batch, hq=hq, hkv=hkv, chunk_lo=rng.randint(1, n), chunk_hi=n, start_hi=start, window=window,
                    softcap=softcap, alibi=rng.random() < 0.5, doc=rng.choice([0, spread(8, 900)]), prefix=rng.choice([0, spread(4, 900)]), out=out)
    rows = spread(1, 2048)
    return dict(op=op, rows=rows, vocab=min(spread(60, 151936), 262668288 // rows), top=rng.choice([0, 1, 5, 20, 32]),
                dtype=rng.choice(["bf16", "fp32"]) if rows <= 1024 else "bf16", scale=rng.choice([1.0, 0.7, 1.4]), masked=rng.random() < 0.3)


def _lengths(n, lo, hi, phase):
    """n lengths over [lo, hi] in no order, the same for every seed; the last one is hi."""
    got = [lo + int((hi - lo) * ((i * 0.6180339887 + phase) % 1.0)) for i in range(n)]
    got[-1] = hi
    return got


def _decode_spans(case):
    """[first visible key, length) of every sequence."""
    lens = _lengths(case["batch"], case["lo"], case["hi"], 0.37)
    first = [int(n * ((i * 0.414213562) % 0.3)) if case["first"] else 0 for i, n in enumerate(lens)]
    lo = [max(f, n - case["window"] if case["window"] else 0, 0) for f, n in zip(first, lens)]
    return lens, first, lo


def _prefill_spans(case):
    """Chunk lengths, cached tokens before them, document lengths and prefixes."""
    n = _lengths(case["batch"], case["chunk_lo"], case["chunk_hi"], 0.23)
    start = _lengths(case["batch"], 0, case["start_hi"], 0.71)
    doc = [max(1, int(case["doc"] * (0.5 + (i * 0.7320508) % 1.0))) if case["doc"] else 0 for i in range(case["batch"])]
    prefix = [int(case["prefix"] * (0.5 + (i * 0.2360679) % 1.0)) for i in range(case["batch"])]
    return n, start, doc, prefix


def _tables_lengths(case):
    start = _lengths(case["batch"], 0 if case["prompts"] else 1, case["context"], 0.11)
    new = [1] * case["batch"]
    for i in range(case["prompts"]):
        new[i * case["batch"] // case["prompts"]] = max(1, case["chunk"] - 7 * i)
    return start, new


def work(case):
    op = case["op"]
    if op == "tables":
        start, new = _tables_lengths(case)
        pages = sum((s + n + 15) // 16 - (s + 15) // 16 for s, n in zip(start, new))
        old = sum(1 for s in start if s % 16)  # entries of pages already begun
        t, b, layers = case["capacity"], case["batch"], case["layers"]
        return {"bytes": 4 * (3 * b + 2 * layers * pages + layers * old + t + layers * t), "flops": 0}
    if op == "rope":
        t, hq, hkv = case["tokens"], case["hq"], case["hkv"]
        rows = min(t, case["context"])
        return {"bytes": t * (128 * (hq + 2 * hkv) + 256 * hq + 128 * 2 * hkv + 8) + rows * case["rot"] * 4,
                "flops": t * (hq + hkv) * case["rot"] * 3}
    if op == "decode":
        lens, _, lo = _decode_spans(case)
        keys = sum(max(n - a, 0) for n, a in zip(lens, lo))
        pages = sum(-(-n // PAGE) - a // PAGE for n, a in zip(lens, lo))
        rows = case["batch"] * case["hq"]
        return {"bytes": keys * case["hkv"] * 256 + rows * 64 * (4 + (2 if case["out"] == "bf16" else 4)) + 4 * pages + 4 * case["batch"],
                "flops": keys * case["hq"] * 256}
    if op == "prefill":
        ns, starts, docs, prefixes = _prefill_spans(case)
        seen = keys = 0
        for n, s, d, p in zip(ns, starts, docs, prefixes):
            low = s + n
            for i in range(s, s + n):
                a = max(i // d * d if d else 0, i - case["window"] + 1 if case["window"] else 0, 0)
                seen += min(max(i + 1, p), s + n) - a
                low = min(low, a)
            keys += s + n - low
        t = sum(ns)
        return {"bytes": keys * case["hkv"] * 256 + t * case["hq"] * 64 * (4 + (2 if case["out"] == "bf16" else 4)),
                "flops": seen * case["hq"] * 256}
    size = 2 if case["dtype"] == "bf16" else 4
    return {"bytes": case["rows"] * (case["vocab"] * size + 12 + 8 * case["top"]), "flops": case["rows"] * case["vocab"] * 6}


# ----------------------------------------------------------------------------
# what a program has in hand before the call


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _normal(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def _frequencies(case):
    """fp64 inverse frequencies of the rotated pairs: plain, linear position
    interpolation, or scaled by wavelength band (long waves slowed by the
    factor, short ones kept, a linear ramp between)."""
    half = case["rot"] // 2
    inv = [500000.0 ** (-2.0 * j / case["rot"]) for j in range(half)]
    if case["scaling"] == "linear":
        inv = [f / 4.0 for f in inv]
    if case["scaling"] == "banded":
        factor, low, high, original = 8.0, 1.0, 4.0, 8192.0
        for j, f in enumerate(inv):
            turns = original * f / (2 * math.pi)
            keep = min(max((turns - low) / (high - low), 0.0), 1.0)
            inv[j] = keep * f + (1 - keep) * f / factor
    return torch.tensor(inv, dtype=torch.float64, device="cuda")


def _rope_table(inv, rows):
    """The framework's cos/sin table of positions 0 .. rows - 1: fp32 pairs
    {cos_hi, cos_lo, sin_hi, sin_lo} of 32 frequencies a row, then {cos, sin} in
    fp64 (frequencies past the rotated ones: angle 0)."""
    angle = torch.zeros(rows, 32, dtype=torch.float64, device="cuda")
    angle[:, : inv.numel()] = torch.arange(rows, device="cuda", dtype=torch.float64)[:, None] * inv
    full = torch.stack([torch.cos(angle), torch.sin(angle)], dim=-1)
    hi = full.float()
    lo = (full - hi.double()).float()
    pairs = torch.stack([hi[..., 0], lo[..., 0], hi[..., 1], lo[..., 1]], dim=-1)
    return torch.cat([pairs.view(torch.uint8).reshape(-1), full.view(torch.uint8).reshape(-1)])


def _pages(g, counts, spare=8):
    """A scattered block table for pages-per-sequence counts: int32 [B][max], and the pool's pages."""
    total = sum(counts)
    perm = torch.randperm(total + spare, generator=g, device="cuda").to(torch.int32)
    cols = max(max(counts), 1)
    at = _ints([sum(counts[:i]) for i in range(len(counts))])[:, None] + torch.arange(cols, device="cuda")[None, :]
    used = torch.arange(cols, device="cuda")[None, :] < _ints(counts)[:, None]
    return torch.where(used, perm[at.clamp(max=total - 1 + spare)], torch.full_like(perm[:1], -1)).contiguous(), total + spare


def _slopes(hq):
    return torch.tensor([2.0 ** (-8.0 * (i + 1) / hq) for i in range(hq)], dtype=torch.float32, device="cuda")


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case)
    if op == "tables":
        start, new = _tables_lengths(case)
        counts = [(n + PAGE - 1) // PAGE for n in start]
        layers, batch = case["layers"], case["batch"]
        cols = max((a + b + PAGE - 1) // PAGE for a, b in zip(start, new))
        held = sum(counts) * layers
        need = sum((a + b + PAGE - 1) // PAGE - c for a, b, c in zip(start, new, counts)) * layers
        pages = held + need + 64
        perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        tables = torch.full((layers, batch, cols), -1, dtype=torch.int32, device="cuda")
        used = torch.arange(cols, device="cuda")[None, :] < _ints(counts)[:, None]
        tables[used.expand(layers, -1, -1)] = perm[:held]
        s.update(start=_ints(start), new=_ints(new), block_tables=tables, free_pages=perm[held:].contiguous(),
                 free_head=_ints([3]), free_head_out=_ints([0]), num_pages=pages,
                 cu_tokens=_ints([0] * (batch + 1)), seq_lens=_ints([0] * batch),
                 positions=_ints([0] * case["capacity"]),
                 slot_map=torch.zeros(layers, case["capacity"], dtype=torch.int32, device="cuda"))
        if own:
            import paged_kv_decode_rope_gb300 as pkv
            s["storage"] = torch.empty(pages * 2 * PAGE * HEAD_DIM, dtype=torch.bfloat16, device="cuda")
            s["pool"] = pkv.kv_pool_create(s["storage"], 1)
        return s
    if op == "rope":
        t, hq, hkv = case["tokens"], case["hq"], case["hkv"]
        pages = -(-t // PAGE) + 4
        # q, k and v are slices of one projection's output
        qkv = _normal(g, t, (hq + 2 * hkv) * HEAD_DIM, scale=1.5)
        q, k, v = qkv.view(t, -1, HEAD_DIM).split([hq, hkv, hkv], dim=1)
        slots = torch.randperm(pages * PAGE, generator=g, device="cuda")[:t].to(torch.int32)
        positions = torch.randint(0, case["context"], (t,), generator=g, device="cuda", dtype=torch.int32)
        s.update(q=q, k=k, v=v, slot_map=slots, positions=positions, table=_rope_table(_frequencies(case), case["context"]),
                 storage=_normal(g, pages, hkv, 2, PAGE, HEAD_DIM),
                 q_rot=torch.empty(t, hq, HEAD_DIM, dtype=torch.float32, device="cuda"))
        if own:
            import paged_kv_decode_rope_gb300 as pkv
            s["pool"] = pkv.kv_pool_create(s["storage"], hkv)
        return s
    if op in ("decode", "prefill"):
        hq, hkv = case["hq"], case["hkv"]
        if op == "decode":
            lens, first, _ = _decode_spans(case)
            rows = case["batch"]
            s.update(seq_lens=_ints(lens), first=_ints(first) if case["first"] else None)
        else:
            chunk, start, doc, prefix = _prefill_spans(case)
            lens = [a + b for a, b in zip(chunk, start)]
            rows = sum(chunk)
            cu = [sum(chunk[:i]) for i in range(len(chunk) + 1)]
            starts = []
            for n, a, d in zip(chunk, start, doc):
                starts += [i // d * d if d else 0 for i in range(a, a + n)]
            s.update(cu_tokens=_ints(cu), start_pos=_ints(start), chunk_hi=max(chunk), len_hi=max(lens),
                     doc_starts=_ints(starts) if case["doc"] else None, prefix_lens=_ints(prefix) if case["prefix"] else None)
        tables, pages = _pages(g, [-(-n // PAGE) for n in lens])
        dtype = torch.bfloat16 if case["out"] == "bf16" else torch.float32
        s.update(block_tables=tables, scale=HEAD_DIM ** -0.5, slopes=_slopes(hq) if case["alibi"] else None,
                 storage=_normal(g, pages, hkv, 2, PAGE, HEAD_DIM),
                 q_rot=torch.randn(rows, hq, HEAD_DIM, generator=g, device="cuda") * 2.0,
                 result=torch.empty(rows, hq, HEAD_DIM, dtype=dtype, device="cuda"))
        if own:
            import paged_kv_decode_rope_gb300 as pkv
            s["pool"] = pkv.kv_pool_create(s["storage"], hkv)
            if op == "decode":
                s["workspace"] = pkv.alloc_decode_workspace(rows, hq, hkv, tables.shape[1])
            else:
                s["workspace"] = pkv.alloc_prefill_workspace(rows, case["batch"], tables.shape[1])
        return s
    rows, vocab, top = case["rows"], case["vocab"], case["top"]
    x = torch.randn(rows, vocab, generator=g, device="cuda") * 2.5
    if case["masked"]:  # a grammar leaves every second row a few tokens
        allowed = torch.rand(rows, vocab, generator=g, device="cuda") < 40.0 / vocab
        x[::2] = torch.where(allowed[::2], x[::2], torch.full_like(x[:1, :1], -math.inf))
    logits = x.to(torch.bfloat16) if case["dtype"] == "bf16" else x
    s.update(logits=logits, targets=torch.randint(0, vocab, (rows,), generator=g, device="cuda", dtype=torch.int32),
             logprobs=torch.empty(rows, dtype=torch.float32, device="cuda"), entropy=torch.empty(rows, dtype=torch.float32, device="cuda"),
             top_ids=torch.empty(rows, top, dtype=torch.int32, device="cuda"),
             top_logprobs=torch.empty(rows, top, dtype=torch.float32, device="cuda"))
    if own:
        import paged_kv_decode_rope_gb300 as pkv
        s["workspace"] = pkv.alloc_logprobs_workspace(rows, vocab, top)
    return s


# ----------------------------------------------------------------------------
# one pass


def run(s):
    op = s["op"]
    if own:
        import paged_kv_decode_rope_gb300 as pkv
        if op == "tables":
            pkv.paged_tables_build(s["pool"], s["start"], s["new"], s["free_pages"], s["free_head"], s["free_head_out"],
                                   s["block_tables"], s["cu_tokens"], s["seq_lens"], s["positions"], s["slot_map"])
        elif op == "rope":
            pkv.paged_rope_append(s["pool"], s["q"], s["k"], s["v"], s["q_rot"], s["slot_map"], s["positions"], s["table"],
                                  rot_dim=s["rot"], interleaved=s["interleaved"])
        elif op == "decode":
            pkv.paged_gqa_decode_scored(s["pool"], s["q_rot"], s["result"], s["block_tables"], s["seq_lens"], s["scale"], s["workspace"],
                                        softcap=s["softcap"], alibi_slopes=s["slopes"], window=s["window"], first_keys=s["first"])
        elif op == "prefill":
            pkv.paged_gqa_prefill_scored(s["pool"], s["q_rot"], s["result"], s["block_tables"], s["cu_tokens"], s["start_pos"], s["scale"],
                                         s["workspace"], softcap=s["softcap"], alibi_slopes=s["slopes"], window=s["window"],
                                         prefix_lens=s["prefix_lens"], doc_starts=s["doc_starts"])
        else:
            pkv.token_logprobs(s["logits"], s["targets"], s["logprobs"], s["entropy"], s["top_ids"], s["top_logprobs"], s["workspace"],
                               scale=s["scale"])
    elif op == "tables":
        _plain_tables(s)
    elif op == "rope":
        _plain_rope(s)
    elif op == "decode":
        _plain_decode(s)
    elif op == "prefill":
        _plain_prefill(s)
    else:
        _plain_logprobs(s)
    if op == "tables":
        return {k: s[k] for k in ("block_tables", "cu_tokens", "seq_lens", "positions", "slot_map", "free_head_out")}
    if op == "rope":
        return {"q_rot": s["q_rot"], "pool": s["storage"]}
    if op in ("decode", "prefill"):
        return s["result"]
    return {k: s[k] for k in ("logprobs", "entropy", "top_ids", "top_logprobs")}


def _plain_tables(s):
    start, new, tables, free = s["start"].long(), s["new"].long(), s["block_tables"], s["free_pages"]
    layers, batch, cols = tables.shape
    capacity, dev = s["capacity"], start.device
    ends = torch.cumsum(new, 0)
    have, want = (start + PAGE - 1) // PAGE, (start + new + PAGE - 1) // PAGE
    ok = (start >= 0) & (new >= 0) & (start + new <= cols * PAGE) & (ends <= capacity)
    need = torch.where(ok, want - have, torch.zeros_like(want))
    base = torch.cumsum(need, 0) - need
    room = (free.numel() - s["free_head"].long()) // layers
    served = ok & ((need == 0) | (base + need <= room))
    need = torch.where(served, need, torch.zeros_like(need))
    # pages in order of sequence, then layer, then block
    col = torch.arange(cols, device=dev)
    fresh = served[:, None] & (col >= have[:, None]) & (col < want[:, None])
    rank = (base * layers)[None, :, None] + torch.arange(layers, device=dev)[:, None, None] * need[None, :, None] + (col - have[:, None])[None]
    page = free[(rank + s["free_head"].long()).clamp(0, free.numel() - 1)]
    tables.copy_(torch.where(fresh[None], page, tables))
    s["cu_tokens"][1:] = ends
    s["seq_lens"].copy_(torch.where(served, start + new, start))
    s["free_head_out"].copy_(s["free_head"] + (need.sum() * layers).to(torch.int32))
    t = torch.arange(capacity, device=dev)
    seq = torch.searchsorted(ends, t, right=True).clamp(max=batch - 1)
    there = (t < ends[-1]) & served[seq]
    pos = torch.where(there, start[seq] + t - (ends - new)[seq], torch.zeros_like(t))
    slot = tables[:, seq, pos // PAGE] * PAGE + (pos % PAGE)[None]
    s["positions"].copy_(pos)
    s["slot_map"].copy_(torch.where(there[None], slot, torch.full_like(slot, -1)))


def _plain_rope(s):
    rot, half, rows = s["rot"], s["rot"] // 2, s["context"]
    full = s["table"][rows * 512:].view(torch.float64).view(rows, 32, 2)
    cs = full[s["positions"].long()][:, None, :half].float()
    cos, sin = cs[..., 0], cs[..., 1]

    def rotate(x):
        x = x.float()
        a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if s["interleaved"] else (x[..., :half], x[..., half:rot])
        y = torch.cat([x[..., :0], a * cos - b * sin, b * cos + a * sin, x[..., rot:]], dim=-1)
        if s["interleaved"]:
            y[..., :rot] = torch.stack([y[..., :half], y[..., half:rot]], dim=-1).flatten(-2)
        return y

    s["q_rot"].copy_(rotate(s["q"]))
    slot = s["slot_map"].long()
    s["storage"][slot // PAGE, :, 0, slot % PAGE] = rotate(s["k"]).to(torch.bfloat16)
    s["storage"][slot // PAGE, :, 1, slot % PAGE] = s["v"]


def _gathered(s):
    """K and V of every sequence's pages, fp32 [B, Hkv, keys, 64]."""
    kv = s["storage"][s["block_tables"].long().clamp(min=0)]  # [B, blocks, Hkv, 2, 16, 64]
    kv = kv.permute(0, 2, 3, 1, 4, 5).flatten(3, 4).float()
    return kv[:, :, 0], kv[:, :, 1]


def _weigh(s, score, key, pos, visible, v):
    """softmax over the visible keys of the capped and biased scores
    [B, Hkv, G, N, keys], times V; rows that see nothing are zero."""
    if s["softcap"]:
        score = s["softcap"] * torch.tanh(score / s["softcap"])
    if s["slopes"] is not None:
        slope = s["slopes"].view(1, s["hkv"], -1, 1, 1)
        score = score - slope * (pos - key).abs()[:, None, None]
    score = torch.where(visible[:, None, None], score, torch.full_like(score[:1, :1, :1, :1, :1], -math.inf))
    top = score.amax(dim=-1, keepdim=True)
    p = torch.exp(score - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = p.sum(dim=-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), v)
    return o.unflatten(2, p.shape[2:4]) / torch.where(total > 0, total, torch.ones_like(total))


def _plain_decode(s):
    k, v = _gathered(s)
    n = s["seq_lens"].long()
    batch, hkv, keys = k.shape[:3]
    key = torch.arange(keys, device=k.device)[None, None, :]
    last = (n - 1)[:, None, None]
    visible = key <= last
    if s["window"]:
        visible = visible & (key > last - s["window"])
    if s["first"] is not None:
        visible = visible & (key >= s["first"][:, None, None])
    q = s["q_rot"].view(batch, hkv, -1, HEAD_DIM)
    score = torch.matmul(q, k.transpose(-1, -2)).unsqueeze(3) * s["scale"]  # [B, Hkv, G, 1, keys]
    v = torch.where(visible[:, :, :, None], v, torch.zeros_like(v[:1, :1, :1]))
    s["result"].copy_(_weigh(s, score, key.float(), last.float(), visible, v).reshape(s["result"].shape))


def _plain_prefill(s):
    k, v = _gathered(s)
    cu, start = s["cu_tokens"].long(), s["start_pos"].long()
    total, width, hkv = s["q_rot"].shape[0], s["chunk_hi"], k.shape[1]
    t = torch.arange(width, device=k.device)
    row = (cu[:-1, None] + t).clamp(max=total - 1)  # [B, N]
    pos = (start[:, None] + t)[:, :, None]
    end = (start + cu[1:] - cu[:-1])[:, None, None]
    key = torch.arange(k.shape[2], device=k.device)[None, None, :]
    visible = key <= pos
    if s["prefix_lens"] is not None:
        visible = visible | (key < s["prefix_lens"][:, None, None])
    visible = visible & (key < end) & (pos < end)
    if s["window"]:
        visible = visible & (key > pos - s["window"])
    if s["doc_starts"] is not None:
        visible = visible & (key >= s["doc_starts"][row][:, :, None])
    q = s["q_rot"][row].unflatten(2, (hkv, -1)).permute(0, 2, 3, 1, 4)  # [B, Hkv, G, N, 64]
    score = torch.matmul(q.flatten(2, 3), k.transpose(-1, -2)).unflatten(2, q.shape[2:4]) * s["scale"]
    v = torch.where((key < end)[:, :, :, None], v, torch.zeros_like(v[:1, :1, :1]))
    o = _weigh(s, score, key.float(), pos.float(), visible, v).permute(0, 3, 1, 2, 4).flatten(2, 3)  # [B, N, Hq, 64]
    at = torch.arange(total, device=k.device)
    seq = torch.searchsorted(cu[1:], at, right=True)
    s["result"].copy_(o[seq, at - cu[seq]])


def _plain_logprobs(s):
    y = s["logits"].float() * s["scale"]
    m = y.amax(dim=-1, keepdim=True)
    z = y - m
    e = torch.exp(z)
    total = e.sum(dim=-1, keepdim=True)
    lse = m + torch.log(total)
    s["logprobs"].copy_((torch.gather(y, 1, s["targets"].long()[:, None]) - lse)[:, 0])
    weighted = torch.where(e > 0, e * z, torch.zeros_like(e)).sum(dim=-1, keepdim=True)
    s["entropy"].copy_((torch.log(total) - weighted / total)[:, 0])
    # the order of the logits as whole numbers, the lower index first among equals
    bits = s["logits"].float().view(torch.int32)
    order = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits).long()
    order = order * 2 ** 24 - torch.arange(y.shape[1], device=y.device)
    ids = torch.topk(order, s["top"], dim=-1, sorted=True).indices
    s["top_ids"].copy_(ids)
    s["top_logprobs"].copy_(torch.gather(y, 1, ids) - lse)


# ----------------------------------------------------------------------------
# the definitions, in 64 bits, one sequence or row at a time


def _exact_attention(s, q, seq, lo, hi, pos, slopes):
    """Attention of the rows q [N, Hq, 64] at positions pos over keys [lo, hi) of sequence seq (lo, hi per row)."""
    keys = int(hi.max())
    pages = s["block_tables"][seq, : -(-keys // PAGE)].long().clamp(min=0)
    kv = s["storage"][pages].double().permute(1, 2, 0, 3, 4).flatten(2, 3)[:, :, :keys]  # [Hkv, 2, keys, 64]
    n, hq, group = q.shape[0], s["hq"], s["hq"] // s["hkv"]
    key = torch.arange(keys, device=q.device)
    seen = (key[None] >= lo[:, None]) & (key[None] < hi[:, None])
    out = torch.zeros(n, hq, HEAD_DIM, dtype=torch.float64, device=q.device)
    some = seen.any(dim=1)
    for h in range(hq):
        x = q[:, h].double() @ kv[h // group, 0].T * s["scale"]
        if s["softcap"]:
            x = s["softcap"] * torch.tanh(x / s["softcap"])
        if slopes is not None:
            x = x - slopes[h].double() * (pos[:, None] - key[None]).abs().double()
        x = x.masked_fill(~seen, -math.inf)
        out[some, h] = torch.softmax(x[some], dim=-1) @ kv[h // group, 1]
    return out


def exact(case, seed):
    op = case["op"]
    if op == "tables":
        return None  # whole numbers
    global own
    was, own = own, False
    s = prepare(case, seed)
    own = was
    if op == "rope":
        angle = s["positions"].double()[:, None] * _frequencies(case)
        turn = torch.polar(torch.ones_like(angle), angle)[:, None]  # cos + i sin, per pair

        def rotate(x):
            r, half = case["rot"], case["rot"] // 2
            y = x.double().clone()
            pair = y[..., :r].unflatten(-1, (half, 2)) if case["interleaved"] else y[..., :r].unflatten(-1, (2, half)).transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
            y[..., :r] = z.flatten(-2) if case["interleaved"] else z.transpose(-1, -2).flatten(-2)
            return y

        pool, at = s["storage"].double(), s["slot_map"].long()
        pool[at // PAGE, :, 0, at % PAGE] = rotate(s["k"])
        pool[at // PAGE, :, 1, at % PAGE] = s["v"].double()
        return {"q_rot": rotate(s["q"]), "pool": pool}
    if op == "decode":
        lens, _, lo = _decode_spans(case)
        return torch.cat([_exact_attention(s, s["q_rot"][b:b + 1], b, _ints([lo[b]]), _ints([n]), _ints([n - 1]), s["slopes"])
                          for b, n in enumerate(lens)])
    if op == "prefill":
        chunk, start, doc, prefix = _prefill_spans(case)
        got, row = [], 0
        for b, (n, a, d, p) in enumerate(zip(chunk, start, doc, prefix)):
            pos = torch.arange(a, a + n, device="cuda")
            lo = pos // d * d if d else torch.zeros_like(pos)
            if case["window"]:
                lo = torch.maximum(lo, pos - case["window"] + 1)
            hi = (pos + 1).clamp(min=p).clamp(max=a + n)
            got.append(_exact_attention(s, s["q_rot"][row:row + n], b, lo, hi, pos, s["slopes"]))
            row += n
        return torch.cat(got)
    x = s["logits"].double() * case["scale"]
    logp = torch.log_softmax(x, dim=-1)
    ids = torch.sort(s["logits"], dim=-1, descending=True, stable=True).indices[:, : case["top"]]
    return {"logprobs": logp[torch.arange(case["rows"], device="cuda"), s["targets"].long()],
            "entropy": torch.special.entr(torch.exp(logp)).sum(dim=-1), "top_ids": None, "top_logprobs": torch.gather(logp, 1, ids)}
