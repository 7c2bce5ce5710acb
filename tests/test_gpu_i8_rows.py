"""The norm and the gated rows with their 8-bit forms on the GPU, against 64-bit arithmetic."""
import numpy as np
import pytest

from tests import i8_helpers as E
from tests.gpu_helpers import to_np

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import heterogeneous_adapter_gemm_amd as hg
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    hg.library()
    yield
    torch.cuda.synchronize()


def say(*a):
    print("[case]", *a, flush=True)


def dev(v):
    return torch.from_numpy(np.asarray(v, np.float32)).to(torch.bfloat16).cuda()


def wide(t, pad):
    """The same rows inside wider ones, 7.0 around them."""
    n, d = t.shape
    big = torch.full((n + 2, d + pad), 7.0, dtype=t.dtype, device=t.device)
    big[1:n + 1, :d] = t
    return big, big[1:n + 1, :d]


def untouched(big, n, d):
    return bool((big[0] == 7.0).all() and (big[n + 1:] == 7.0).all() and (big[:, d:] == 7.0).all())


def outputs(n, d, pad=8):
    y, held = (wide(torch.full((n, d), 7.0, dtype=torch.bfloat16, device="cuda"), pad) for _ in range(2))
    code = torch.full((n + 1, d), 77, dtype=torch.int8, device="cuda")
    scale = torch.full((n + 1,), 7.0, device="cuda")
    return y, held, code, scale


def check_form(code, scale, held, want_code, want_scale, rel, n):
    assert np.array_equal(code[:n].cpu().numpy().astype(np.float64), want_code)
    s = scale[:n].double().cpu().numpy()
    assert np.all(np.abs(s - want_scale) <= want_scale * rel + E.TINY)
    if held is not None:
        v = want_code * s[:, None]
        assert np.all(np.abs(to_np(held) - v) <= np.abs(v) * (E.HALF + 2 * E.ULP) + E.TINY)


# widths of every kind of row: 16, 32 and 64 lanes' (one and two vectors a lane), a workgroup's with 1, 2, 3, 4 and 8
WIDTHS = [8, 64, 72, 128, 136, 256, 264, 512, 520, 1024, 1032, 4096, 4104, 5120, 8192, 8200, 11008, 12288, 12296, 16384, 16392, 28672, 65536]


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("n,with_residual", [(1, True), (5, False), (9, True)])
def test_norm(d, n, with_residual):
    import heterogeneous_adapter_gemm_amd as hg
    say("norm", n, d, with_residual)
    g = np.random.default_rng(n * 100003 + d)
    ch = np.exp(0.7 * g.standard_normal(d))
    x, w = E.bf16(g.standard_normal((n, d)) * ch), E.bf16(1 + 0.2 * g.standard_normal(d))
    res = E.bf16(2 * g.standard_normal((n, d)) * ch) if with_residual else None
    x[0, d // 2] = 0.5 * x[0, 0]
    eps = [1e-5, 1e-6][n % 2]
    _, xd = wide(dev(x), 16)
    rd = wide(dev(res), 24)[1] if with_residual else None
    (yb, y), (hb, held), code, scale = outputs(n, d)
    sb, s = wide(torch.full((n, d), 7.0, dtype=torch.bfloat16, device="cuda"), 32)
    hg.rows_norm_i8(xd, dev(w), eps, residual=rd, sum_out=s if with_residual else None, y=y, code=code[:n], scale=scale[:n], held=held)
    torch.cuda.synchronize()
    h, want, want_code, want_scale = E.norm(x, res, w, eps)
    if with_residual:
        assert np.array_equal(to_np(s), h)
    # the sum of squares: a thread adds up to 64 of them, then 6 steps of a wave and 16 waves; half of that in the
    # root, which with the quotients and factors adds 8 roundings
    rel = (0.5 * (64 + 6 + 16 + 2) + 8) * E.ULP
    assert np.all(np.abs(to_np(y) - want) <= np.abs(want) * (E.HALF + rel) + E.TINY)
    check_form(code, scale, held, want_code, want_scale, rel, n)
    assert untouched(yb, n, d) and untouched(hb, n, d) and untouched(sb, n, d)
    assert bool((code[n] == 77).all()) and float(scale[n]) == 7.0


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("act,n", [("silu", 3), ("gelu", 5), ("gelu_tanh", 1), ("none", 6)])
def test_act(d, act, n):
    import heterogeneous_adapter_gemm_amd as hg
    say("act", act, n, d)
    g = np.random.default_rng(n * 100003 + d)
    gate, x = E.bf16(3 * g.standard_normal((n, d))), E.bf16(g.standard_normal((n, d)))
    gate[0, :8] = [-100, -20, -9.5, -1e-3, 0, 1e-3, 30, 100]
    both = dev(np.concatenate([gate, x], 1))      # as one projection's output
    (yb, y), (hb, held), code, scale = outputs(n, d)
    hg.rows_act_i8(both[:, d:], gate=None if act == "none" else both[:, :d], act=act, y=y, code=code[:n], scale=scale[:n], held=held)
    torch.cuda.synchronize()
    a = to_np(y)
    if act == "none":
        assert np.array_equal(a, x)
    else:
        assert np.all(np.abs(a - E.activated(gate, act) * x) <= E.act_bound(act, gate, x))
    # the form is that of the bf16 rows
    check_form(code, scale, held, E.codes(a), np.abs(a).max(1) / 127, E.ULP, n)
    assert untouched(yb, n, d) and untouched(hb, n, d)
    assert bool((code[n] == 77).all()) and float(scale[n]) == 7.0


@pytest.mark.parametrize("size", [2.0 ** -125, 2.0 ** -90, 2.0 ** -30, 1.0, 2.0 ** 30, 2.0 ** 59])
def test_sizes_and_ties(size):
    """Codes of rows whose quotients fall on ties, from the least normal numbers up to squares near fp32's end."""
    import heterogeneous_adapter_gemm_amd as hg
    d = 1024
    g = np.random.default_rng(7)
    x = np.concatenate([g.integers(-127, 128, (3, d)), 2 * g.integers(-63, 64, (3, d)) + 1]).astype(np.float64)
    x[:, 0] = [254, 127, 128, 254, 127, 126]
    x = E.bf16(x * size / 256)
    w = np.ones(d)
    code = torch.zeros((6, d), dtype=torch.int8, device="cuda")
    scale, y = torch.zeros(6, device="cuda"), torch.zeros((6, d), dtype=torch.bfloat16, device="cuda")
    hg.rows_act_i8(dev(x), code=code, scale=scale)
    torch.cuda.synchronize()
    check_form(code, scale, None, E.codes(x), np.abs(x).max(1) / 127, E.ULP, 6)
    hg.rows_norm_i8(dev(x), dev(w), 1e-30, y=y, code=code, scale=scale)
    torch.cuda.synchronize()
    _, want, want_code, want_scale = E.norm(x, None, w, float(np.float32(1e-30)))
    check_form(code, scale, None, want_code, want_scale, 60 * E.ULP, 6)
    assert np.all(np.abs(to_np(y) - want) <= np.abs(want) * (E.HALF + 60 * E.ULP) + E.TINY)


@pytest.mark.parametrize("d", [64, 1000, 4096, 11008])
def test_rows_of_zeros_and_rows_that_are_not_finite(d):
    import heterogeneous_adapter_gemm_amd as hg
    g = np.random.default_rng(d)
    n = 7
    x, w = E.bf16(g.standard_normal((n, d))), E.bf16(1 + 0.2 * g.standard_normal(d))
    clean = dev(x)
    bad = clean.clone()
    bad[1] = 0
    bad[2, d - 1], bad[4, 0], bad[5, d // 2] = np.inf, np.nan, -np.inf
    got = []
    for rows in (clean, bad):
        (_, y), (_, held), code, scale = outputs(n, d)
        hg.rows_norm_i8(rows, dev(w), 1e-5, y=y, code=code[:n], scale=scale[:n], held=held)
        ya, ha, ca, sa = (torch.zeros_like(t) for t in (y, held, code[:n], scale[:n]))
        hg.rows_act_i8(rows, gate=torch.ones_like(rows), act="silu", y=ya, code=ca, scale=sa, held=ha)
        torch.cuda.synchronize()
        got.append([t.float().cpu().numpy() for t in (y, held, code[:n], scale[:n], ya, ha, ca, sa)])
    for k, (a, b) in enumerate(zip(*got)):
        assert np.array_equal(a[[0, 3, 6]], b[[0, 3, 6]]), k
        assert not np.any(b[1]), k
        if k in (2, 6):                     # codes
            assert not np.any(b[[2, 4, 5]])
        elif k != 4:                        # (y of the gated rows is NaN or infinite where its value is)
            assert np.all(np.isnan(b[[2, 4, 5]])), k


def test_squares_past_the_range_are_nan():
    import heterogeneous_adapter_gemm_amd as hg
    x = torch.full((2, 512), 2.0 ** 62, dtype=torch.bfloat16, device="cuda")
    x[1] = 2.0 ** 55
    y, code, scale = torch.zeros_like(x), torch.zeros((2, 512), dtype=torch.int8, device="cuda"), torch.zeros(2, device="cuda")
    hg.rows_norm_i8(x, torch.ones(512, dtype=torch.bfloat16, device="cuda"), 1e-5, y=y, code=code, scale=scale)
    assert bool(torch.isnan(y[0]).all()) and bool(torch.isnan(scale[0])) and bool((y[1] == 1).all()) and bool((code[1] == 127).all())


@pytest.mark.parametrize("d", [8, 136, 4096, 65536])
def test_products_past_the_range(d):
    """Squares that fit, times a weight that does not: infinities in y, and no codes; the rows beside are not touched by it."""
    import heterogeneous_adapter_gemm_amd as hg
    x = torch.ones((3, d), dtype=torch.bfloat16, device="cuda")
    x[1, d - 1] = 2.0 ** 50
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    w[d - 1] = 2.0 ** 100
    y, held = torch.zeros_like(x), torch.zeros_like(x)
    code, scale = torch.full((3, d), 5, dtype=torch.int8, device="cuda"), torch.zeros(3, device="cuda")
    hg.rows_norm_i8(x, w, 1e-5, y=y, code=code, scale=scale, held=held)
    torch.cuda.synchronize()
    assert bool(torch.isinf(y[1, d - 1])) and bool(torch.isfinite(y[1, :d - 1]).all()) and bool(torch.isfinite(y[0]).all())
    assert bool(torch.isnan(scale[1])) and bool((code[1] == 0).all()) and bool(torch.isnan(held[1]).all())
    for t in (0, 2):
        assert int(code[t, d - 1]) == 127 and bool((code[t, :d - 1] == 0).all()) and bool(torch.isfinite(scale[t]))


@pytest.mark.parametrize("d", [64, 4096])
def test_some_outputs_only_and_in_place(d):
    import heterogeneous_adapter_gemm_amd as hg
    g = np.random.default_rng(d)
    n = 11
    x, r, w = (dev(g.standard_normal(s)) for s in ((n, d), (n, d), (d,)))
    full = [torch.zeros((n, d), dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    code, scale = torch.zeros((n, d), dtype=torch.int8, device="cuda"), torch.zeros(n, device="cuda")
    hg.rows_norm_i8(x, w, 1e-5, residual=r, sum_out=full[0], y=full[1], held=full[2], code=code, scale=scale)
    y1, h1, c1, s1 = (torch.zeros_like(t) for t in (full[1], full[2], code, scale))
    hg.rows_norm_i8(x, w, 1e-5, residual=r, y=y1)
    hg.rows_norm_i8(x, w, 1e-5, residual=r, held=h1)
    hg.rows_norm_i8(x, w, 1e-5, residual=r, code=c1, scale=s1)
    a, b = x.clone(), r.clone()
    hg.rows_norm_i8(a, w, 1e-5, residual=b, sum_out=b, y=a)
    torch.cuda.synchronize()
    for got, want in ((y1, full[1]), (h1, full[2]), (c1, code), (s1, scale), (b, full[0]), (a, full[1])):
        assert torch.equal(got, want)
    y2, h2 = torch.zeros_like(x), torch.zeros_like(x)
    hg.rows_act_i8(x, gate=r, act="gelu", y=y2, held=h2, code=code, scale=scale)
    c2, s2, a, b = torch.zeros_like(code), torch.zeros_like(scale), x.clone(), r.clone()
    hg.rows_act_i8(x, gate=r, act="gelu", code=c2, scale=s2)
    hg.rows_act_i8(a, gate=b, act="gelu", y=a, held=b)
    torch.cuda.synchronize()
    for got, want in ((c2, code), (s2, scale), (a, y2), (b, h2)):
        assert torch.equal(got, want)


def test_many_rows():
    """More rows than a round of workgroups; odd counts of a wave's rows; the norm's wave a row."""
    import heterogeneous_adapter_gemm_amd as hg
    for n, d in ((20003, 128), (9001, 1032), (4001, 200), (2049, 2048), (2500, 2056), (2048, 4096), (3001, 4104)):
        say("many rows", n, d)
        g = np.random.default_rng(n)
        x = E.bf16(g.standard_normal((n, d)))
        w = E.bf16(1 + 0.2 * g.standard_normal(d))
        (_, y), (_, held), code, scale = outputs(n, d)
        hg.rows_norm_i8(dev(x), dev(w), 1e-5, y=y, code=code[:n], scale=scale[:n], held=held)
        torch.cuda.synchronize()
        _, want, want_code, want_scale = E.norm(x, None, w, 1e-5)
        assert np.all(np.abs(to_np(y) - want) <= np.abs(want) * (E.HALF + 60 * E.ULP) + E.TINY)
        check_form(code, scale, held, want_code, want_scale, 60 * E.ULP, n)


def test_captured_and_on_another_stream():
    import heterogeneous_adapter_gemm_amd as hg
    g = np.random.default_rng(1)
    n, d = 33, 2048
    x, r, w = (dev(g.standard_normal(s)) for s in ((n, d), (n, d), (d,)))
    outs = [torch.zeros((n, d), dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    code, scale, c2, s2 = (torch.zeros(s, dtype=t, device="cuda") for s, t in (((n, d), torch.int8), ((n,), torch.float32)) * 2)

    def step():
        hg.rows_norm_i8(x, w, 1e-5, residual=r, sum_out=outs[0], y=outs[1], code=code, scale=scale)
        hg.rows_act_i8(outs[1], gate=outs[0], act="silu", y=outs[2], code=c2, scale=s2)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    other = torch.cuda.Stream()
    for _ in range(3):
        x.copy_(dev(g.standard_normal((n, d))))
        graph.replay()
        torch.cuda.synchronize()
        want = [t.clone() for t in (*outs, code, scale, c2, s2)]
        for t in (*outs, code, scale, c2, s2):
            t.zero_()
        other.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(other):
            step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (*outs, code, scale, c2, s2)))
