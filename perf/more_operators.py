"""The operators of a layer served in 8-bit integers, measured: the norm of a residual stream with
its 8-bit form, the 8-bit form of (gated) rows, the product of 8-bit rows with an 8-bit weight, alone
and with adapters, and the gated product of a feed-forward block.

Each is given twice: in elementary torch operations, and (where ``own`` is true) as the calls of this
repository's package.  The 8-bit form of a row is scale * code, code -127..127 the nearest integers to
127 * row / max|row| (ties to even), scale one fp32 number a row; of a weight, one scale an output
channel.  ``held`` rows are what the codes stand for, rounded to bf16.
"""
import math
import random

import torch

own = False

EPS = 1e-5


# -- cases ------------------------------------------------------------------------------------

def listed():
    return [
        # one token of a lone request: latency is all
        dict(name="norm one row", op="norm", rows=1, d=4096, residual=True),
        # the rows of the stack step between two blocks
        dict(name="norm stack", op="norm", rows=2961, d=4096, residual=True),
        # a decode step's gate and up rows on their way into the down projection
        dict(name="act decode 64", op="act", rows=64, d=11008, act="silu", merged=True),
        # the stack step's
        dict(name="act stack", op="act", rows=2961, d=11008, act="silu", merged=False),
        # a lone token through a square projection
        dict(name="product one row", op="product", rows=1, n=4096, k=4096),
        # 64 decode rows through the up projection
        dict(name="product decode 64", op="product", rows=64, n=11008, k=4096),
        # 256 decode rows through the down projection
        dict(name="product decode 256", op="product", rows=256, n=4096, k=11008),
        # the stack step's rows through a square projection
        dict(name="product stack", op="product", rows=2961, n=4096, k=4096),
        # the decode layer with adapters: 64 rows over 16 adapters of rank 16
        dict(name="linear decode 64", op="linear", rows=64, n=4096, k=4096, segs=0, adapters=16, rank=16),
        # the stack step's mix: 8 prompts and 192 decode rows, each with an adapter of its own choice
        dict(name="linear stack", op="linear", rows=2961, n=4096, k=4096, segs=8, adapters=24, rank=32),
        # gate and up of 64 decode rows in one
        dict(name="gated decode 64", op="gated", rows=64, n=11008, k=4096, act="silu"),
        # gate and up of the stack step
        dict(name="gated stack", op="gated", rows=2961, n=11008, k=4096, act="silu"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


ACTS = ("silu", "gelu", "gelu_tanh")


def draw(rng):
    op = rng.choice(["norm", "norm", "act", "act", "product", "product", "product", "linear", "linear", "gated"])
    if op == "norm":
        d = 8 * _log(rng, 8, 2048)
        return dict(op=op, rows=_log(rng, 1, max(2, min(20000, 24_000_000 // d))), d=d, residual=rng.random() < 0.7)
    if op == "act":
        d = 8 * _log(rng, 8, 4096)
        act = rng.choice(ACTS + ("none",))
        return dict(op=op, rows=_log(rng, 1, max(2, min(20000, 32_000_000 // d))), d=d, act=act,
                    merged=act != "none" and rng.random() < 0.5)
    rows = _log(rng, 1, 3000)
    n = 8 * _log(rng, 8, 1400)
    k = 16 * _log(rng, 8, 700)
    if op == "product":
        return dict(op=op, rows=rows, n=n, k=k)
    if op == "gated":
        return dict(op=op, rows=rows, n=n, k=k, act=rng.choice(ACTS))
    segs = 0 if rows < 128 else rng.randint(1, 9)
    return dict(op=op, rows=rows, n=n, k=k, segs=segs, adapters=rng.randint(1, 24), rank=rng.choice([4, 8, 16, 33, 64]))


def work(case):
    T = case["rows"]
    if case["op"] == "norm":
        # x, the residual and the weight read; their sum, the normed rows, the codes and what they stand for written
        n = T * case["d"]
        return {"bytes": n * (2 + (4 if case["residual"] else 0) + 2 + 1 + 2) + 2 * case["d"] + 4 * T, "flops": 10 * n}
    if case["op"] == "act":
        n = T * case["d"]
        return {"bytes": n * ((2 if case["act"] == "none" else 6) + 1 + 2) + 4 * T, "flops": 16 * n}
    N, K = case["n"], case["k"]
    if case["op"] == "gated":
        return {"bytes": 2 * N * (K + 4) + T * (K + 4) + 2 * T * N, "flops": 4 * T * N * K}
    w = {"bytes": N * (K + 4) + T * (K + 4) + 2 * T * N, "flops": 2 * T * N * K}
    if case["op"] == "linear":
        w["bytes"] += min(T, case["adapters"]) * case["rank"] * (N + K) * 2 + 2 * T * K
        w["flops"] += 2 * T * case["rank"] * (N + K)
    return w


# -- inputs -----------------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _rows(case, seed):
    """The bf16 rows a call reads: (x, residual or gate or None, weight or None)."""
    g = _gen(seed)
    T = case["rows"]
    if case["op"] == "norm":
        d = case["d"]
        wide = torch.exp(0.7 * _normal(g, d))                     # a residual stream: some channels are far wider
        x = (_normal(g, T, d) * 0.5 * wide).to(torch.bfloat16)
        r = (_normal(g, T, d) * 2.0 * wide).to(torch.bfloat16) if case["residual"] else None
        return x, r, (1.0 + 0.2 * _normal(g, d)).to(torch.bfloat16)
    if case["op"] == "act":
        d = case["d"]
        x = (_normal(g, T, d) * 0.9).to(torch.bfloat16)
        gate = None if case["act"] == "none" else (_normal(g, T, d) * 1.7).to(torch.bfloat16)
        return x, gate, None
    return (_normal(g, T, case["k"]) * torch.exp(0.4 * _normal(g, case["k"]))).to(torch.bfloat16), None, None


def _eight(x):
    """The 8-bit form of rows: int8 codes and fp32 scales, in 64 bits up to the rounding."""
    x = x.double()
    most = x.abs().amax(-1, keepdim=True)
    code = torch.where(most > 0, x * 127.0 / torch.where(most > 0, most, torch.ones_like(most)), torch.zeros_like(x))
    return torch.round(code).to(torch.int8), (most[..., 0] / 127.0).float()


def _weight(case, seed, which):
    """An 8-bit weight: codes [n, k] int8, scales [n]."""
    g = _gen(seed + 10 + which)
    code = (_normal(g, case["n"], case["k"]) * 30.0).round().clamp(-127, 127).to(torch.int8)
    return code, torch.rand(case["n"], generator=g, device="cuda") * 1e-3 + 2e-4


def _split(case):
    """Row starts of the prompts; the rows behind them are decode rows."""
    r = random.Random(case["rows"] * 31 + case["segs"])
    pre = case["rows"] - case["rows"] // 16 if case["segs"] else 0
    cut = sorted(r.randint(0, pre) for _ in range(case["segs"] - 1)) if case["segs"] else []
    return [0] + cut + [pre] if case["segs"] else [0]


def _adapters(case, seed):
    """A [n, rank, K], B [n, rank, N] bf16 on the host, alpha per adapter, the adapter of each prompt and
    decode row, and of every row (-1 = none)."""
    g = torch.Generator().manual_seed(seed + 3)
    n, r = case["adapters"], case["rank"]
    A = (torch.randn((n, r, case["k"]), generator=g) * case["k"] ** -0.5).to(torch.bfloat16)
    B = (torch.randn((n, r, case["n"]), generator=g) * 0.02).to(torch.bfloat16)
    alpha = [2.0 * r + i for i in range(n)]
    st = _split(case)
    seg = torch.randint(-1, n, (case["segs"],), generator=g, dtype=torch.int32)
    dec = torch.randint(-1, n, (case["rows"] - st[-1],), generator=g, dtype=torch.int32)
    lens = torch.tensor([b - a for a, b in zip(st, st[1:])], dtype=torch.int64)
    who = torch.cat([torch.repeat_interleave(seg, lens), dec]) if case["segs"] else dec
    return A, B, alpha, st, seg, dec, who


def prepare(case, seed):
    s = {"case": case}
    T = case["rows"]
    x, other, w = _rows(case, seed)
    if case["op"] in ("norm", "act"):
        d = case["d"]
        if case.get("merged"):      # gate and up side by side, as one projection writes them
            both = torch.cat([other, x], 1)
            other, x = both[:, :d], both[:, d:]
        s["x"], s["other"], s["w"] = x, other, w
        empty = lambda dtype: torch.zeros((T, d), dtype=dtype, device="cuda")  # noqa: E731
        s["sum"] = empty(torch.bfloat16) if case["op"] == "norm" and case["residual"] else None
        s["y"] = None if case.get("act") == "none" else empty(torch.bfloat16)
        s["held"], s["code"] = empty(torch.bfloat16), empty(torch.int8)
        s["scale"] = torch.zeros(T, device="cuda")
        return s
    s["code"], s["scale"] = _eight(x)
    s["w"] = [_weight(case, seed, i) for i in range(2 if case["op"] == "gated" else 1)]
    s["y"] = torch.zeros((T, case["n"]), dtype=torch.bfloat16, device="cuda")
    if case["op"] == "linear":
        A, B, alpha, st, seg, dec, who = _adapters(case, seed)
        s["x"], s["A"], s["B"], s["who"] = x, A.cuda(), B.cuda(), who.cuda()
        s["gamma"] = torch.tensor([a / case["rank"] for a in alpha], device="cuda")
        if own:
            import heterogeneous_adapter_gemm_amd as hg
            n, r, P = case["adapters"], case["rank"], 4096
            need = n * r * (-(-case["k"] // P) - (-case["n"] // P))
            pool = hg.DevicePool(hg.LORA_BF16, P, need + 8, None, 1, [case["k"]], [case["n"]], n + 1, 64, T,
                                 max(case["segs"], 1))
            for i in range(n):
                pool.page_in_pinned(i, r, alpha[i], A[i].flatten().pin_memory(), B[i].flatten().pin_memory())
                torch.cuda.synchronize()
            s["pool"] = pool
            s["plan"] = pool.plan(st, pool.slots_of(seg.numpy()), pool.slots_of(dec.numpy())) if case["segs"] else \
                pool.plan(token_slot=pool.slots_of(dec.numpy()))
    return s


# -- the operators ----------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    return run_norm(s) if op == "norm" else run_act(s) if op == "act" else run_product(s)


def _form(p):
    """Codes (as 32-bit numbers) and greatest magnitude of rows p; the quotients in 64 bits, next to a
    rounding's border a code has to fall on one side."""
    most = p.abs().amax(-1, keepdim=True)
    safe = torch.where(most > 0, most, torch.ones_like(most))
    return torch.round(p.double() * 127.0 / safe.double()).float(), most


def run_norm(s):
    if own:
        import heterogeneous_adapter_gemm_amd as hg
        hg.rows_norm_i8(s["x"], s["w"], EPS, residual=s["other"], sum_out=s["sum"], y=s["y"], code=s["code"],
                        scale=s["scale"], held=s["held"])
        return {"sum": s["sum"], "y": s["y"], "held": s["held"], "scale": s["scale"]}
    h = s["x"] if s["other"] is None else (s["x"].float() + s["other"].float()).to(torch.bfloat16)
    f = h.float()
    r = 1.0 / torch.sqrt((f * f).mean(-1, keepdim=True) + EPS)
    p = f * s["w"].float()
    code, most = _form(p)
    scale = most * r / 127.0
    return {"sum": None if s["other"] is None else h, "y": (p * r).to(torch.bfloat16),
            "held": (code * scale).to(torch.bfloat16), "scale": scale[:, 0]}


def _activated(x, act):
    if act == "silu":
        return x / (1.0 + torch.exp(-x))
    if act == "gelu":
        return 0.5 * x * torch.erfc(x * -math.sqrt(0.5))
    return x / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (x + 0.044715 * x * x * x)))


def run_act(s):
    act = s["case"]["act"]
    if own:
        import heterogeneous_adapter_gemm_amd as hg
        hg.rows_act_i8(s["x"], gate=s["other"], act=act, y=s["y"], code=s["code"], scale=s["scale"], held=s["held"])
        return {"y": s["y"], "held": s["held"], "scale": s["scale"]}
    a = s["x"] if act == "none" else (_activated(s["other"].float(), act) * s["x"].float()).to(torch.bfloat16)
    code, most = _form(a.float())
    scale = most / 127.0
    return {"y": None if act == "none" else a, "held": (code * scale).to(torch.bfloat16), "scale": scale[:, 0]}


def run_product(s):
    case = s["case"]
    T, N, K = case["rows"], case["n"], case["k"]
    if own:
        import heterogeneous_adapter_gemm_amd as hg
        if case["op"] == "product":
            hg.base_gemm_i8(s["code"], s["scale"], *s["w"][0], s["y"], T, N, K)
        elif case["op"] == "gated":
            hg.base_gated_i8(s["code"], s["scale"], *s["w"][0], *s["w"][1], s["y"], T, N, K, act=case["act"])
        else:
            s["pool"].linear_i8(s["plan"], 0, 0, s["x"], s["code"], s["scale"], *s["w"][0], s["y"])
        return s["y"]
    x = s["code"].float()
    product = lambda w: torch.matmul(x, w[0].float().t()) * s["scale"][:, None] * w[1]  # noqa: E731
    y = product(s["w"][0])
    if case["op"] == "gated":
        y = _activated(y, case["act"]) * product(s["w"][1])
    if case["op"] == "linear":
        who = s["who"].long()
        mid = torch.matmul(s["x"].float(), s["A"].float().flatten(0, 1).t()).unflatten(-1, s["A"].shape[:2])    # [T, n, r]
        mine = (torch.arange(s["A"].shape[0], device="cuda")[None] == who[:, None]).float()
        mid = mid * (mine * s["gamma"][None])[..., None]
        y = y + torch.matmul(mid.flatten(1), s["B"].float().flatten(0, 1))
    return y.to(torch.bfloat16)


# -- in 64 bits, from the definitions --------------------------------------------------------

def _exact_held(v):
    """What the 8-bit form of rows v stands for, and its scale."""
    scale = v.abs().max(-1, keepdim=True).values / 127
    return (v / torch.where(scale > 0, scale, 1.0)).round() * scale, scale[:, 0]


def _exact_act(v, act):
    if act == "silu":
        return v * torch.special.expit(v)
    if act == "gelu":
        return v * torch.special.ndtr(v)
    return 0.5 * v * (1 + torch.tanh((2 / math.pi) ** 0.5 * (v + 0.044715 * v ** 3)))


def exact(case, seed):
    x, other, w = _rows(case, seed)
    if case["op"] == "norm":
        h = x.double()
        if other is not None:
            h = (h + other.double()).float().to(torch.bfloat16).double()      # the stream itself is kept in bf16
        n = h * torch.rsqrt(h.pow(2).mean(-1, keepdim=True) + EPS) * w.double()
        held, scale = _exact_held(n)
        return {"sum": None if other is None else h, "y": n, "held": held, "scale": scale}
    if case["op"] == "act":
        a = x.double()
        if other is not None:
            a = _exact_act(other.double(), case["act"]) * a
        held, scale = _exact_held(a.float().to(torch.bfloat16).double())      # the 8-bit form is that of the bf16 rows
        return {"y": None if other is None else a, "held": held, "scale": scale}
    code, scale = _eight(x)
    left = code.double() * scale.double()[:, None]
    def product(which):
        c, s = _weight(case, seed, which)
        return left @ (c.double() * s.double()[:, None]).t().contiguous()
    y = product(0)
    if case["op"] == "gated":
        return _exact_act(y, case["act"]) * product(1)
    if case["op"] == "linear":
        A, B, alpha, _, _, _, who = _adapters(case, seed)
        xd = x.double()
        for a in range(case["adapters"]):
            mine = (who == a).nonzero().flatten().cuda()
            if mine.numel():
                y[mine] += alpha[a] / case["rank"] * ((xd[mine] @ A[a].cuda().double().t().contiguous()) @ B[a].cuda().double())
    return y
