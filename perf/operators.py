"""The operators of a 4-bit served attention block, measured: the base product over a 4-bit
weight, the append of a step's keys and values to the pool's KV pages (4 bits, the position
rotation on the way), and attention over those pages.

Each is given twice: in elementary torch operations, and (where ``own`` is true) as the calls
of this repository's package.  Layouts both read and write:

  4-bit rows of the KV pages: a row of head_dim values stands for lo + step * code, code
  0..15, with one 32-bit word per row (bf16 step in the low half, bf16 lo in the high half).
  16 consecutive tokens of one KV head's keys (or values) are one slab of 8 head_dim + 64
  bytes: the codes, then the 16 words.  Slab 2 h is head h's keys, 2 h + 1 its values; a
  block of 16 tokens takes ceil(2 heads / (page bytes / slab bytes)) pages.
  Key codes: token-major; in each 32-bit word of 8 values, nibble k is value 2 k and nibble
  k + 4 value 2 k + 1.  Value codes: for i in 0..15 the head_dim / 16 values from
  i head_dim / 16 on: [i][token pair][4 values][token of the pair], 16 bits each.

  4-bit weights: W[n][k] = scale * (code - zero), byte k / 2 of row n holding code k in its
  low (even k) or high half, scale and zero fp16 per ``group`` consecutive k.
"""
import math
import random

import torch

own = False

BLOCK = 16


# -- cases ------------------------------------------------------------------------------------

def listed():
    return [
        # one decode step's new rows of 64 requests, 32 query heads over 8 KV heads
        dict(name="append decode 64", op="append", seqs=64, lo=128, hi=4096, rows=1, heads=32, kv_heads=8, dim=128,
             rot=128, interleaved=False, page=4096, shape=1),
        # one layer of the 32-head, 4096-wide stack step: 8 prompts of 128..512 tokens
        dict(name="append prompts stack", op="append", seqs=8, lo=128, hi=512, rows=-1, heads=32, kv_heads=32, dim=128,
             rot=128, interleaved=False, page=4096, shape=2),
        # a lone request answered token by token: latency is all
        dict(name="attend one request", op="attend", seqs=1, lo=1000, hi=1000, rows=1, heads=32, kv_heads=8, dim=128,
             page=4096, shape=3),
        # a serving step: 64 requests of very different lengths
        dict(name="attend decode 64", op="attend", seqs=64, lo=128, hi=4096, rows=1, heads=32, kv_heads=8, dim=128,
             page=4096, shape=4),
        # the decode rows of the stack step: 192 requests, as many KV heads as query heads
        dict(name="attend decode stack", op="attend", seqs=192, lo=129, hi=552, rows=1, heads=32, kv_heads=32, dim=128,
             page=4096, shape=5),
        # one long document: the split over the tokens
        dict(name="attend long", op="attend", seqs=1, lo=131071, hi=131071, rows=1, heads=32, kv_heads=8, dim=128,
             page=4096, shape=6),
        # three drafted tokens a request checked at once, one shared KV head, narrow heads
        dict(name="attend drafts", op="attend", seqs=33, lo=200, hi=3001, rows=3, heads=12, kv_heads=1, dim=64, page=1024,
             shape=7),
        # prompts taken in pieces: 512 rows behind up to 4096 tokens each
        dict(name="attend prompt pieces", op="attend", seqs=4, lo=512, hi=4096, rows=512, heads=32, kv_heads=8, dim=128,
             page=4096, shape=8),
        # a lone token through a 4096 x 4096 projection
        dict(name="base one row", op="base", rows=1, n=4096, k=4096, group=128),
        # 64 decode rows through the up projection
        dict(name="base decode 64", op="base", rows=64, n=11008, k=4096, group=128),
        # the decode layer with adapters: 64 rows over 16 adapters of rank 16
        dict(name="linear decode 64", op="linear", rows=64, n=4096, k=4096, group=128, adapters=16, rank=16),
        # the stack step's 2,961 rows through a square projection
        dict(name="base stack", op="base", rows=2961, n=4096, k=4096, group=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "attend", "attend", "attend", "base", "base", "linear"])
    if op in ("append", "attend"):
        dim = rng.choice([64, 128, 128, 256])
        kv_heads = rng.choice([1, 2, 3, 8, 16])
        heads = kv_heads * rng.choice([1, 2, 4, 5, 8])
        page = rng.choice([4096, 8192] if dim > 128 else [1024, 4096, 16384])
        kind = rng.choice(["decode", "drafts", "pieces"])
        seqs = _log(rng, 1, 8 if kind == "pieces" else 96)
        rows = 1 if kind == "decode" else rng.randint(2, 9) if kind == "drafts" else _log(rng, 20, 400)
        # (at most about 40 MB of cache, or 8,000 rows times tokens a head)
        most = max(16, min(60000, 40_000_000 // (seqs * kv_heads * dim)))
        hi = max(rows, _log(rng, 16, most if kind != "pieces" else min(most, 4000)))
        case = dict(op=op, seqs=seqs, lo=max(1, hi // rng.choice([1, 2, 20])), hi=hi, rows=rows, heads=heads,
                    kv_heads=kv_heads, dim=dim, page=page, shape=rng.randrange(1 << 30))
        if op == "append":
            case["rot"] = rng.choice([dim, dim, dim // 2, 32])
            case["interleaved"] = rng.random() < 0.5
        return case
    group = rng.choice([32, 64, 128])
    rows = _log(rng, 1, 600)
    n = 4 * _log(rng, 32, 2800 if rows < 200 else 1200)
    k = 128 * rng.randint(1, 40)
    case = dict(op=op, rows=rows, n=n, k=k, group=group)
    if op == "linear":
        case["n"] = n - n % 8 + 8
        case["adapters"] = rng.randint(1, 24)
        case["rank"] = rng.choice([4, 8, 16, 33, 64])
    return case


def _lengths(case):
    """Rows of this step and tokens in the cache after it, per request."""
    r = random.Random(case["shape"])
    tokens = [r.randint(case["lo"], case["hi"]) for _ in range(case["seqs"])]
    if case["rows"] < 0:    # whole prompts
        return list(tokens), tokens
    return [min(case["rows"], t) for t in tokens], tokens


def _slab(dim):
    return 8 * dim + 64


def _geometry(case):
    slabs = 2 * case["kv_heads"]
    per_page = 2 * case["page"] // _slab(case["dim"])
    return slabs, per_page, -(-slabs // per_page)


def work(case):
    if case["op"] in ("append", "attend"):
        rows, tokens = _lengths(case)
        T, D, H, KV = sum(rows), case["dim"], case["heads"], case["kv_heads"]
        if case["op"] == "append":
            # q, k, v read and written as bf16, the rows' codes and words, the table's rows
            return {"bytes": T * D * 2 * 2 * (H + 2 * KV) + T * 2 * KV * (D // 2 + 4) + sum(rows) * case["rot"] * 4,
                    "flops": 3 * T * (H + KV) * case["rot"] + 6 * T * 2 * KV * D}
        seen = sum(sum(t - n + 1 + j for j in range(n)) for n, t in zip(rows, tokens))
        return {"bytes": sum(tokens) * 2 * KV * (D // 2 + 4) + 2 * T * H * D * 2, "flops": 4 * seen * H * D}
    M, N, K = case["rows"], case["n"], case["k"]
    w = {"bytes": N * K // 2 + N * (K // case["group"]) * 4 + 2 * M * (N + K), "flops": 2 * M * N * K}
    if case["op"] == "linear":
        w["bytes"] += min(M, case["adapters"]) * case["rank"] * (N + K) * 2
        w["flops"] += 2 * M * case["rank"] * (N + K)
    return w


# -- inputs -----------------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _quantise(x):
    """bf16 rows [..., D] -> (codes 0..15, bf16 step, bf16 lo) of the 4-bit rows."""
    h = x.float() * 0.5
    lo, hi = h.amin(-1), h.amax(-1)
    step = ((hi - lo) / 7.5).to(torch.bfloat16)
    lo = x.amin(-1)
    half = step.float() * 0.5
    safe = torch.where(half > 0, half, torch.ones_like(half))
    t = torch.round((h - lo.float()[..., None] * 0.5) / safe[..., None]).clamp(0, 15)
    code = torch.where((half > 0)[..., None], t, torch.zeros_like(t))
    return code.to(torch.int32), step, lo


def _words(step, lo):
    bits = lambda t: t.view(torch.int16).to(torch.int32) & 0xFFFF  # noqa: E731
    return bits(step) | (bits(lo) << 16)


def _key_bytes(code):
    """codes [..., 16, D] -> the slab's key bytes [..., 8 D]."""
    c = code.unflatten(-1, (-1, 4, 2)).transpose(-1, -2).flatten(-2)        # nibble order of each word
    return (c[..., 0::2] | (c[..., 1::2] << 4)).to(torch.uint8).flatten(-3)


def _value_bytes(code):
    """codes [..., 16, D] -> the slab's value bytes [..., 8 D]."""
    D = code.shape[-1]
    c = code.unflatten(-1, (16, D // 64, 4)).unflatten(-4, (8, 2))          # [.., pair, token, i, part, 4]
    c = c.movedim(-3, -5).movedim(-3, -2)                                   # [.., i, pair, part, token, 4]
    return (c[..., 0::2] | (c[..., 1::2] << 4)).to(torch.uint8).flatten(-5)


def _slabs(k, v):
    """keys and values as (codes [B, 16, H, D], step, lo [B, 16, H]) -> slab bytes [B, 2 H, slab]."""
    def one(x, pack):
        code, step, lo = x
        words = _words(step, lo).transpose(1, 2).contiguous().view(torch.uint8)             # [B, H, 64]
        return torch.cat([pack(code.transpose(1, 2)), words], -1)
    return torch.stack([one(k, _key_bytes), one(v, _value_bytes)], 2).flatten(1, 2)


def _cache_rows(case, seed):
    """Every cached token's keys and values as bf16 rows [requests * most blocks * 16, heads, D]."""
    g = _gen(seed)
    _, tokens = _lengths(case)
    nb = -(-max(tokens) // BLOCK)
    shape = (case["seqs"] * nb * BLOCK, case["kv_heads"], case["dim"])
    spread = torch.exp(0.5 * _normal(g, case["kv_heads"], case["dim"]))     # some channels are wider
    k = (_normal(g, *shape) * spread + _normal(g, case["kv_heads"], case["dim"])).to(torch.bfloat16)
    v = (_normal(g, *shape) * 0.7).to(torch.bfloat16)
    return k, v


def _pages_of(case, seed):
    """A pool's pages in a shuffled physical order, every byte 0xFF, and the batch's page table."""
    _, per_page, npb = _geometry(case)
    _, tokens = _lengths(case)
    blocks = [-(-t // BLOCK) for t in tokens]
    total = sum(blocks) * npb
    page_bytes = 2 * case["page"]
    pages = torch.full((total + 7, page_bytes), 255, dtype=torch.uint8, device="cuda")
    order = torch.randperm(total + 7, generator=torch.Generator().manual_seed(seed))[:total].to(torch.int32)
    table = torch.full((case["seqs"], max(blocks), npb), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(blocks):
        table[s, :n] = order[at:at + n * npb].view(n, npb)
        at += n * npb
    return pages, table.cuda()


def _handle(case, pages):
    """The pool a program keeps; its pages hold the prepared ones."""
    import heterogeneous_adapter_gemm_amd as hg
    pool = hg.DevicePool(hg.LORA_BF16, case["page"], pages.shape[0], None, 1, [512], [512], 1, 8, 64, 1)
    pool.pages.view(torch.uint8).copy_(pages.flatten())
    return pool


def prepare(case, seed):
    if case["op"] in ("base", "linear"):
        return _prepare_base(case, seed)
    s = {"case": case}
    rows, tokens = _lengths(case)
    T, D = sum(rows), case["dim"]
    g = _gen(seed + 1)
    s["rows"], s["tokens"], s["T"] = rows, tokens, T
    starts = [0]
    for n in rows:
        starts.append(starts[-1] + n)
    s["row_start"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    s["ctx_len"] = torch.tensor(tokens, dtype=torch.int32, device="cuda")
    pages, table = _pages_of(case, seed)
    s["table"] = table
    s["q"] = (_normal(g, T, case["heads"], D) * 1.3).to(torch.bfloat16)
    if case["op"] == "append":
        s["k"] = _normal(g, T, case["kv_heads"], D).to(torch.bfloat16)
        s["v"] = _normal(g, T, case["kv_heads"], D).to(torch.bfloat16)
        half = case["rot"] // 2
        pos = torch.arange(table.shape[1] * BLOCK, dtype=torch.float64, device="cuda")
        freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
        ang = pos[:, None] * freq
        s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float()
        s["q_out"], s["k_out"], s["v_out"] = (torch.zeros_like(s[n]) for n in ("q", "k", "v"))
    else:
        _, per_page, npb = _geometry(case)
        nb = table.shape[1]
        k, v = _cache_rows(case, seed)
        cut = lambda x: [t.view(-1, BLOCK, *t.shape[1:]) for t in _quantise(x)]  # noqa: E731
        slabs = _slabs(cut(k), cut(v))
        del k, v
        full = torch.zeros((slabs.shape[0], npb * per_page, slabs.shape[2]), dtype=torch.uint8, device="cuda")
        full[:, :slabs.shape[1]] = slabs
        full = full.view(case["seqs"], nb, npb, per_page * slabs.shape[2])
        # tokens behind a request's end keep the words of 0xFF bytes (not a number)
        used = torch.arange(nb * BLOCK, device="cuda")[None] < s["ctx_len"][:, None]
        w = full.view(case["seqs"], nb, npb * per_page, -1)[:, :, :slabs.shape[1], 8 * D:].view(torch.int32)
        w.masked_fill_(~used.view(case["seqs"], nb, 1, BLOCK), -1)
        at = table >= 0
        pages[table[at].long(), :full.shape[-1]] = full[at]
        s["out"] = torch.zeros_like(s["q"])
    s["pages"] = pages
    if own:
        import heterogeneous_adapter_gemm_amd as hg
        s["pool"] = _handle(case, pages)
        s["batch"] = hg.KvBatch(case["heads"], case["kv_heads"], D, s["row_start"], s["ctx_len"], table, T,
                                max_rows=max(rows))
        if case["op"] == "attend":
            s["workspace"] = s["pool"].kv_workspace(s["batch"])
    return s


def _weights(case, seed):
    """codes [N, K] int32, scale and zero [N, K / group] fp16."""
    g = _gen(seed + 2)
    N, K, G = case["n"], case["k"], case["group"]
    code = torch.randint(0, 16, (N, K), generator=g, device="cuda", dtype=torch.uint8)
    scale = (torch.rand((N, K // G), generator=g, device="cuda") * 0.006 + 0.002).half()
    zero = torch.randint(5, 11, (N, K // G), generator=g, device="cuda").half()
    return code, scale, zero


def _adapters(case, seed):
    """A [n, rank, K], B [n, rank, N] bf16 on the host, alpha per adapter, the rows' adapters (-1 = none)."""
    g = torch.Generator().manual_seed(seed + 3)
    n, r = case["adapters"], case["rank"]
    A = (torch.randn((n, r, case["k"]), generator=g) * case["k"] ** -0.5).to(torch.bfloat16)
    B = (torch.randn((n, r, case["n"]), generator=g) * 0.02).to(torch.bfloat16)
    alpha = [2.0 * r + i for i in range(n)]
    who = torch.randint(-1, n, (case["rows"],), generator=g, dtype=torch.int32)
    return A, B, alpha, who


def _rows_of_x(case, seed):
    return _normal(_gen(seed), case["rows"], case["k"]).to(torch.bfloat16)


def _prepare_base(case, seed):
    s = {"case": case, "x": _rows_of_x(case, seed)}
    code, scale, zero = _weights(case, seed)
    s["code"] = (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous()
    s["scale"] = torch.stack([scale, zero], -1).contiguous()
    s["y"] = torch.zeros((case["rows"], case["n"]), dtype=torch.bfloat16, device="cuda")
    if case["op"] == "linear":
        A, B, alpha, who = _adapters(case, seed)
        s["A"], s["B"], s["who"] = A.cuda(), B.cuda(), who.cuda()
        s["gamma"] = torch.tensor([a / case["rank"] for a in alpha], device="cuda")
        if own:
            import heterogeneous_adapter_gemm_amd as hg
            n, r, P = case["adapters"], case["rank"], 4096
            need = n * r * (-(-case["k"] // P) - (-case["n"] // P))
            pool = hg.DevicePool(hg.LORA_BF16, P, need + 8, None, 1, [case["k"]], [case["n"]], n + 1, 64,
                                 max(case["rows"], 1), 1)
            for i in range(n):
                pool.page_in_pinned(i, r, alpha[i], A[i].flatten().pin_memory(), B[i].flatten().pin_memory())
                torch.cuda.synchronize()
            s["pool"] = pool
            s["plan"] = pool.plan(token_slot=pool.slots_of(who.numpy()))
    return s


# -- the operators ----------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if op == "append":
        return run_append(s)
    if op == "attend":
        return run_attend(s)
    return run_base(s)


def run_append(s):
    case = s["case"]
    if own:
        s["pool"].kv_append(s["batch"], s["k"], s["v"], q=s["q"], q_out=s["q_out"], k_out=s["k_out"], v_out=s["v_out"],
                            cos_sin=s["cos_sin"], interleaved=case["interleaved"])
        return s["q_out"], s["k_out"], s["v_out"]
    t = torch.arange(s["T"], device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["row_start"], t, right=True) - 1
    pos = (s["ctx_len"][seq] - s["row_start"][seq + 1] + t).long()
    cos, sin = s["cos_sin"][pos].double().chunk(2, -1)
    q = _rotate(s["q"], cos, sin, case)
    k = _rotate(s["k"], cos, sin, case)
    code_k, step_k, lo_k = _quantise(k)
    code_v, step_v, lo_v = _quantise(s["v"])
    _store(s, seq, pos, (code_k, step_k, lo_k), (code_v, step_v, lo_v))
    value = lambda c, st, lo: (lo.float()[..., None] + st.float()[..., None] * c).to(torch.bfloat16)  # noqa: E731
    return q, value(code_k, step_k, lo_k), value(code_v, step_v, lo_v)


def _rotate(x, cos, sin, case):
    """Pairs (i, i + rot / 2), or (2 i, 2 i + 1) when interleaved, of the first rot values turned by
    their angle, in 64 bits: a key next to a rounding's border has to fall on one side of it."""
    rot = case["rot"]
    d = x[..., :rot].double()
    a, b = (d[..., 0::2], d[..., 1::2]) if case["interleaved"] else d.chunk(2, -1)
    c, s = cos[:, None], sin[:, None]
    a, b = a * c - b * s, b * c + a * s
    r = torch.stack([a, b], -1).flatten(-2) if case["interleaved"] else torch.cat([a, b], -1)
    return torch.cat([r.float().to(torch.bfloat16), x[..., rot:]], -1)


def _store(s, seq, pos, k, v):
    """The rows' codes and words to their places in the pages."""
    case = s["case"]
    D, KV = case["dim"], case["kv_heads"]
    slabs, per_page, npb = _geometry(case)
    flat = s["pages"].view(-1)
    block, r = (pos // BLOCK), (pos % BLOCK)
    slab = torch.arange(slabs, device="cuda")
    page = s["table"][seq[:, None], block[:, None], (slab // per_page)[None]].long()
    base = page * (2 * case["page"]) + (slab % per_page) * _slab(D)          # [T, 2 KV]
    kb, vb = base[:, 0::2], base[:, 1::2]

    def nibbles(c):     # [.., 8] in nibble order -> bytes
        return (c[..., 0::2] | (c[..., 1::2] << 4)).to(torch.uint8)

    kc = k[0].unflatten(-1, (-1, 4, 2)).transpose(-1, -2).flatten(-2)
    at = kb[..., None] + r[:, None, None] * (D // 2) + torch.arange(D // 2, device="cuda")
    flat[at.flatten()] = nibbles(kc).flatten()
    vc = nibbles(v[0].unflatten(-1, (16, D // 64, 4)))                        # [T, KV, i, part, 2]
    i = torch.arange(16, device="cuda")[:, None, None] * (D // 2)
    part = torch.arange(D // 64, device="cuda")[None, :, None] * 4
    byte = torch.arange(2, device="cuda")[None, None]
    place = i + part + byte + ((r // 2) * (D // 16) + (r % 2) * 2)[:, None, None, None]
    flat[(vb[..., None, None, None] + place[:, None]).flatten()] = vc.flatten()
    words = torch.stack([_words(*k[1:]), _words(*v[1:])], -1).flatten(1)      # [T, 2 KV]
    flat.view(torch.int32)[((base + 8 * D) // 4 + r[:, None]).flatten()] = words.flatten()


def _scale(case):
    return case["dim"] ** -0.5


def run_attend(s):
    case = s["case"]
    if own:
        s["pool"].kv_attention(s["batch"], s["q"], s["out"], scale=_scale(case), workspace=s["workspace"])
        return s["out"]
    D, KV, H = case["dim"], case["kv_heads"], case["heads"]
    slabs, per_page, npb = _geometry(case)
    n, nb = s["table"].shape[:2]
    got = s["pages"][s["table"].clamp(min=0).long()]                          # [n, nb, npb, page bytes]
    got = got[..., :per_page * _slab(D)].reshape(n, nb, npb * per_page, _slab(D))[:, :, :slabs]
    live = torch.arange(nb * BLOCK, device="cuda")[None] < s["ctx_len"][:, None]                  # [n, L]
    k = _unpack(got[:, :, 0::2], live, D, True)                               # [n, KV, L, D] fp32
    v = _unpack(got[:, :, 1::2], live, D, False)
    most = int(max(s["rows"]))
    j = torch.arange(most, device="cuda")
    count = (s["row_start"][1:] - s["row_start"][:-1])[:, None]
    row = (s["row_start"][:-1, None] + j).long()                              # [n, most]
    real = j[None] < count
    q = s["q"][row.clamp(max=s["T"] - 1)].float()                             # [n, most, H, D]
    q = q.view(n, most, KV, H // KV, D).permute(0, 2, 3, 1, 4).reshape(n, KV, -1, D)
    limit = s["ctx_len"][:, None] - count + 1 + j[None]                       # tokens a row sees
    see = torch.arange(nb * BLOCK, device="cuda")[None, None] < limit[..., None]
    see = (see & live[:, None]).repeat(1, H // KV, 1)[:, None]                # [n, 1, G most, L]
    score = torch.matmul(q, k.transpose(-1, -2).contiguous()) * _scale(case)
    score = torch.where(see, score, torch.full_like(score, -math.inf))
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, torch.ones_like(total))
    o = o.view(n, KV, H // KV, most, D).permute(0, 3, 1, 2, 4).reshape(n, most, H, D)
    out = torch.zeros_like(s["q"])
    out[row[real]] = o[real].to(torch.bfloat16)
    return out


def _unpack(slab, live, D, keys):
    """slab bytes [n, nb, KV, slab] -> the values they stand for [n, KV, L, D] in 32 bits."""
    n, nb, KV, _ = slab.shape
    b = slab[..., :8 * D].to(torch.int32)
    c = torch.stack([b & 15, b >> 4], -1).flatten(-2)                         # nibbles [.., 16 D]
    if keys:
        c = c.unflatten(-1, (BLOCK, D // 8, 2, 4)).transpose(-1, -2).flatten(-3)                  # [.., 16, D]
    else:
        c = c.unflatten(-1, (16, 8, D // 64, 2, 4)).permute(0, 1, 2, 4, 6, 3, 5, 7).reshape(n, nb, KV, BLOCK, D)
    w = slab[..., 8 * D:].contiguous().view(torch.int32)                      # [n, nb, KV, 16]
    step = (w << 16).view(torch.float32)
    lo = (w & -65536).view(torch.float32)
    x = lo[..., None] + step[..., None] * c
    x = x.permute(0, 2, 1, 3, 4).reshape(n, KV, nb * BLOCK, D)
    return torch.where(live[:, None, :, None], x, torch.zeros_like(x))


def run_base(s):
    case = s["case"]
    if own:
        import heterogeneous_adapter_gemm_amd as hg
        if case["op"] == "linear":
            s["pool"].linear_w4(s["plan"], 0, 0, s["x"], s["code"], s["scale"], case["group"], s["y"])
        else:
            hg.base_gemm_w4(s["x"], s["code"], s["scale"], s["y"], case["rows"], case["n"], case["k"], case["group"])
        return s["y"]
    code = torch.stack([s["code"] & 15, s["code"] >> 4], -1).flatten(-2).float()
    scale, zero = s["scale"].float().unbind(-1)
    w = (code.unflatten(-1, (-1, case["group"])) - zero[..., None]) * scale[..., None]
    x = s["x"].float()
    y = torch.matmul(x, w.flatten(-2).t())
    if case["op"] == "linear":
        who = s["who"].long()
        a = who.clamp(min=0)
        mid = torch.matmul(x, s["A"].float().flatten(0, 1).t()).unflatten(-1, s["A"].shape[:2])    # [T, n, r]
        mine = (torch.arange(s["A"].shape[0], device="cuda")[None] == who[:, None]).float()
        mid = mid * (mine * s["gamma"][None])[..., None]
        y = y + torch.matmul(mid.flatten(1), s["B"].float().flatten(0, 1))
    return y.to(torch.bfloat16)


# -- in 64 bits, from the definitions --------------------------------------------------------

def exact(case, seed):
    """What run() returns, computed in 64 bits request by request (or product by product) from the
    rows themselves: no pages, no packed codes."""
    if case["op"] == "append":
        return _exact_append(case, seed)
    if case["op"] == "attend":
        return _exact_attend(case, seed)
    x = _rows_of_x(case, seed).double()
    code, scale, zero = _weights(case, seed)
    per = lambda t: t.double().repeat_interleave(case["group"], 1)  # noqa: E731
    y = x @ ((code.double() - per(zero)) * per(scale)).t().contiguous()
    if case["op"] == "linear":
        A, B, alpha, who = _adapters(case, seed)
        for a in range(case["adapters"]):
            mine = (who == a).nonzero().flatten().cuda()
            if mine.numel():
                y[mine] += alpha[a] / case["rank"] * ((x[mine] @ A[a].cuda().double().t().contiguous()) @ B[a].cuda().double())
    return y


def _exact_row4(x):
    """The values the 4-bit form of bf16 rows x stands for, in 64 bits (step and lo are bf16)."""
    x = x.double()
    lo, hi = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
    step = ((hi - lo) / 15).float().to(torch.bfloat16).double()
    code = torch.where(step > 0, ((x - lo) / torch.where(step > 0, step, 1.0)).round().clamp(0, 15), 0.0)
    return lo + step * code


def _exact_append(case, seed):
    rows, tokens = _lengths(case)
    T, D, rot = sum(rows), case["dim"], case["rot"]
    g = _gen(seed + 1)
    q = (_normal(g, T, case["heads"], D) * 1.3).to(torch.bfloat16).double()
    k = _normal(g, T, case["kv_heads"], D).to(torch.bfloat16).double()
    v = _normal(g, T, case["kv_heads"], D).to(torch.bfloat16)
    half = rot // 2
    pos = torch.cat([torch.arange(t - n, t) for n, t in zip(rows, tokens)]).double().cuda()
    freq = torch.pow(torch.tensor(10000.0, dtype=torch.float64, device="cuda"),
                     -torch.arange(half, device="cuda").double() / half)
    turn = torch.complex((pos[:, None] * freq).cos().float().double(), (pos[:, None] * freq).sin().float().double())
    def rotated(x):
        y = x.clone()
        first = slice(0, rot, 2) if case["interleaved"] else slice(0, half)
        second = slice(1, rot, 2) if case["interleaved"] else slice(half, rot)
        z = torch.complex(x[..., first], x[..., second]) * turn[:, None]
        y[..., first], y[..., second] = z.real, z.imag
        return y
    # (a cached key is the 4-bit form of the bf16 key)
    return rotated(q), _exact_row4(rotated(k).float().to(torch.bfloat16)), _exact_row4(v)


def _exact_attend(case, seed):
    rows, tokens = _lengths(case)
    D, KV, H = case["dim"], case["kv_heads"], case["heads"]
    q = (_normal(_gen(seed + 1), sum(rows), H, D) * 1.3).to(torch.bfloat16).double()
    k, v = _cache_rows(case, seed)
    most = -(-max(tokens) // BLOCK) * BLOCK
    out, at = [], 0
    for i, (n, t) in enumerate(zip(rows, tokens)):
        kk, vv = (_exact_row4(x[i * most:i * most + t]).transpose(0, 1).contiguous() for x in (k, v))    # [KV, t, D]
        for h in range(KV):
            qq = q[at:at + n, h * (H // KV):(h + 1) * (H // KV)]             # [n, G, D]
            s = (qq.reshape(-1, D) @ kk[h].t().contiguous()).view(n, -1, t) * _scale(case)
            late = torch.arange(t, device="cuda")[None] > (t - n + torch.arange(n, device="cuda"))[:, None]
            s = s.masked_fill(late[:, None], -math.inf)
            out.append((torch.softmax(s, -1).reshape(-1, t) @ vv[h]).view(n, -1, D))
        at += n
    per, o = [], 0
    for _ in rows:
        per.append(torch.cat(out[o:o + KV], 1))
        o += KV
    return torch.cat(per)
