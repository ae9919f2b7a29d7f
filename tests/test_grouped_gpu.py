"""Grouped products (bf16 forward, gradient of the rows and of the weights,
and the 8-bit form with block scales) against the same sums in 64 bits.

Tolerances: products of bf16 (and of e4m3) values are exact in fp32.  A tensor
core adds 16 (32) of them to a running fp32 sum and cuts what does not fit:
each addition costs at most a step, 2^-23, of a partial sum that the sum of
the magnitudes bounds, and so does each of the additions of partial sums and
scales.  Over a reduction of length n that is (n / 16 + 64) 2^-23 of the sum
of magnitudes, plus half a step of the output type."""
import pytest
import torch

from gpu_util import requires_gpu

pytestmark = [pytest.mark.gpu, requires_gpu]

STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
NAN = float("nan")


def _rn(g, *shape, dt=torch.bfloat16, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dt)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _offsets(counts, first=0):
    o = [first]
    for n in counts:
        o.append(o[-1] + n)
    return torch.tensor(o, dtype=torch.int32, device="cuda"), o


def _check(got, ref, mag, length):
    tol = STEP[got.dtype] * ref.abs() + (length / 16 + 64) * 2.0 ** -23 * mag
    bad = (got.double() - ref).abs() - tol
    assert torch.all(bad <= 0), (float(bad.max()), float((got.double() - ref).abs().max()))


# group sizes (0: an expert without rows), N, K
SHAPES = [
    ([1], 8, 8),
    ([3], 136, 64),
    ([0, 1, 0, 17, 2, 0], 264, 200),
    ([130, 0, 1, 257, 16, 64], 136, 264),
    ([300], 1000, 72),
    ([1] * 8 + [0] * 24, 512, 1024),
    ([65, 700, 0, 33], 328, 2056),
    ([40] * 20, 128, 128),
    ([513], 256, 6144),
    ([2048, 5], 520, 136),
    # more than a wave of narrow tiles: wide ones, in pairs of CTAs
    ([65, 700, 0, 33, 2], 1608, 1544),
    ([3000], 520, 200),
    ([2048, 5, 9], 776, 1000),
    ([513], 2312, 6144),
]


@pytest.mark.parametrize("out_dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("counts,N,K", SHAPES)
def test_forward_and_gradients(counts, N, K, out_dt):
    from int4_routed_expert_coli_b200 import coli_moe as c
    E = len(counts)
    first, behind = 3, 5     # rows of no expert around the groups
    off, o = _offsets(counts, first)
    R = o[-1] + behind
    g = _gen(N * 31 + K)
    x, w, dy = _rn(g, R, K), _rn(g, E, N, K, scale=0.1), _rn(g, R, N)
    # rows of no group may hold anything
    for t in (x, dy):
        t[:first] = NAN
        t[o[-1]:] = float("inf")
    ws = c.grouped_workspace(R, E)
    for repeat in range(2):  # the second call finds the workspace as the first left it
        out = torch.full((R, N), NAN, dtype=out_dt, device="cuda")
        dx = torch.full((R, K), NAN, dtype=out_dt, device="cuda")
        dw = torch.full((E, N, K), NAN, dtype=out_dt, device="cuda")
        c.coli_moe_grouped_mm(R, E, N, K, x, w, off, out, ws)
        c.coli_moe_grouped_mm_dx(R, E, N, K, dy, w, off, dx, ws)
        c.coli_moe_grouped_mm_dw(R, E, N, K, dy, x, off, dw, False, ws)
        assert c.coli_moe_get_status(ws) == c.COLI_OK
    for t in (out, dx):
        assert torch.isnan(t[:first]).all() and torch.isnan(t[o[-1]:]).all()
    for e in range(E):
        lo, hi = o[e], o[e + 1]
        X, W, D = x[lo:hi].double(), w[e].double(), dy[lo:hi].double()
        _check(out[lo:hi], X @ W.T, X.abs() @ W.abs().T, K)
        _check(dx[lo:hi], D @ W, D.abs() @ W.abs(), N)
        _check(dw[e], D.T @ X, D.abs().T @ X.abs(), hi - lo)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_weight_gradient_accumulates(dt):
    from int4_routed_expert_coli_b200 import coli_moe as c
    counts, N, K = [70, 0, 5], 200, 136
    off, o = _offsets(counts)
    R, E = o[-1], len(counts)
    g = _gen(1)
    x, dy = _rn(g, R, K), _rn(g, R, N)
    ws = c.grouped_workspace(R, E)
    dw = _rn(g, E, N, K, dt=dt)
    old = dw.double()
    c.coli_moe_grouped_mm_dw(R, E, N, K, dy, x, off, dw, True, ws)
    for e in range(E):
        X, D = x[o[e]:o[e + 1]].double(), dy[o[e]:o[e + 1]].double()
        _check(dw[e], old[e] + D.T @ X, old[e].abs() + D.abs().T @ X.abs(), 70)
    assert torch.equal(dw[1].double(), old[1])


def test_one_infinite_row_stays_in_its_group():
    """The last K-block of a group ends inside the next group's rows: what they
    hold does not enter its weight gradient."""
    from int4_routed_expert_coli_b200 import coli_moe as c
    counts, N, K = [37, 3, 60], 128, 192
    off, o = _offsets(counts)
    R, E = o[-1], 3
    g = _gen(2)
    x, dy = _rn(g, R, K), _rn(g, R, N)
    x[38] = float("inf")
    dy[39] = NAN
    dw = torch.empty(E, N, K, device="cuda")
    c.coli_moe_grouped_mm_dw(R, E, N, K, dy, x, off, dw, False, c.grouped_workspace(R, E))
    for e in (0, 2):
        X, D = x[o[e]:o[e + 1]].double(), dy[o[e]:o[e + 1]].double()
        _check(dw[e], D.T @ X, D.abs().T @ X.abs(), 64)
    assert not torch.isfinite(dw[1]).any()


def _quantize(t):
    """e4m3 and scales [R][blocks] by the definition, in 64 bits except the
    scale and the quotient (fp32 numbers by definition)."""
    R, K = t.shape
    kb = -(-K // 128)
    pad = torch.zeros(R, kb * 128, dtype=torch.float64, device=t.device)
    pad[:, :K] = t.double()
    b = pad.view(R, kb, 128)
    s = (b.abs().amax(2) / 448.0).float().clamp_min(2.0 ** -126)
    q = (b / s.double()[:, :, None]).float().to(torch.float8_e4m3fn)
    return q.view(R, -1)[:, :K].contiguous(), s


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R,K", [(1, 16), (3, 128), (9, 272), (130, 2048), (17, 6144), (5, 1296)])
def test_quantize_rows(R, K, dt):
    from int4_routed_expert_coli_b200 import coli_moe as c
    g = _gen(R + K)
    x = _rn(g, R, K, dt=dt, scale=3.0)
    x[0, :16] = 0
    if R > 1:
        x[1] = 0                                   # a row of zeros
        x[2, :128] = 2.0 ** -130 if dt == torch.float32 else 2.0 ** -126   # subnormal quotient's scale
    q = torch.empty(R, K, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.full((-(-K // 128), R), NAN, device="cuda")
    c.coli_moe_fp8_quantize_rows(R, K, x, q, s)
    rq, rs = _quantize(x)
    assert torch.equal(s, rs.T.contiguous())
    assert torch.equal(q.view(torch.uint8), rq.view(torch.uint8))


def test_quantize_keeps_infinity_and_nan_visible():
    from int4_routed_expert_coli_b200 import coli_moe as c
    R, K = 3, 256
    x = torch.ones(R, K, device="cuda", dtype=torch.bfloat16)
    x[0, 3] = float("inf")
    x[1, 200] = NAN
    q = torch.empty(R, K, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty(2, R, device="cuda")
    c.coli_moe_fp8_quantize_rows(R, K, x, q, s)
    assert torch.isinf(s[0, 0]) and torch.isfinite(s[1, 0])
    assert torch.isnan(s[1, 1]) and torch.isfinite(s[0, 1])
    assert torch.all(s[:, 2] == 1.0 / 448.0) and torch.all(q[2].float() == 448.0)
    N, E = 16, 1
    wq = torch.ones(E, N, K, device="cuda").to(torch.float8_e4m3fn)
    sw = torch.ones(E, 1, 2, device="cuda")
    off = torch.tensor([0, R], dtype=torch.int32, device="cuda")
    out = torch.empty(R, N, device="cuda")
    c.coli_moe_fp8_grouped_mm(R, E, N, K, q, s, wq, sw, off, out, c.grouped_workspace(R, E))
    assert torch.isnan(out[:2]).all()
    assert torch.all((out[2] - K).abs() <= K * 2.0 ** -20)


@pytest.mark.parametrize("out_dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("counts,N,K", [(s, n, -(-k // 16) * 16) for s, n, k in SHAPES])
def test_fp8_forward(counts, N, K, out_dt):
    from int4_routed_expert_coli_b200 import coli_moe as c
    E = len(counts)
    first, behind = 2, 3
    off, o = _offsets(counts, first)
    R = o[-1] + behind
    g = _gen(N * 37 + K)
    nb, kb = -(-N // 128), -(-K // 128)
    x = _rn(g, R, K)
    wq = _rn(g, E, N, K, dt=torch.float32, scale=100.0).clamp(-448, 448).to(torch.float8_e4m3fn)
    sw = torch.rand(E, nb, kb, generator=g, device="cuda") * 1e-3 + 1e-4
    xq = torch.empty(R, K, dtype=torch.float8_e4m3fn, device="cuda")
    sx = torch.empty(kb, R, device="cuda")
    c.coli_moe_fp8_quantize_rows(R, K, x, xq, sx)
    out = torch.full((R, N), NAN, dtype=out_dt, device="cuda")
    ws = c.grouped_workspace(R, E)
    for repeat in range(2):
        c.coli_moe_fp8_grouped_mm(R, E, N, K, xq, sx, wq, sw, off, out, ws)
        assert c.coli_moe_get_status(ws) == c.COLI_OK
    X = xq.double() * sx.T.double().repeat_interleave(128, 1)[:, :K]
    assert torch.isnan(out[:first]).all() and torch.isnan(out[o[-1]:]).all()
    for e in range(E):
        lo, hi = o[e], o[e + 1]
        W = wq[e].double() * sw[e].double().repeat_interleave(128, 0)[:N] \
            .repeat_interleave(128, 1)[:, :K]
        _check(out[lo:hi], X[lo:hi] @ W.T, X[lo:hi].abs() @ W.abs().T, K)


def test_bad_offsets_are_reported_and_skipped():
    """Groups that descend or leave the rows: nothing is read or written for
    them, the others are right."""
    from int4_routed_expert_coli_b200 import coli_moe as c
    R, E, N, K = 40, 5, 64, 64
    g = _gen(5)
    x, w, dy = _rn(g, R, K), _rn(g, E, N, K), _rn(g, R, N)
    # [0, 10) good, [10, 5) descends, [5, 90) leaves the rows, [90, 20) descends, [20, 40) good
    off = torch.tensor([0, 10, 5, 90, 20, 40], dtype=torch.int32, device="cuda")
    ws = c.grouped_workspace(R, E)
    out = torch.full((R, N), 7.0, device="cuda")
    c.coli_moe_grouped_mm(R, E, N, K, x, w, off, out, ws)
    assert c.coli_moe_get_status(ws) == c.COLI_ERR_BAD_INDEX
    assert torch.all(out[10:20] == 7.0)
    _check(out[:10], x[:10].double() @ w[0].double().T, x[:10].double().abs() @ w[0].double().abs().T, K)
    _check(out[20:], x[20:].double() @ w[4].double().T, x[20:].double().abs() @ w[4].double().abs().T, K)
    c.coli_moe_workspace_clear(ws)
    dw = torch.full((E, N, K), 7.0, device="cuda")
    c.coli_moe_grouped_mm_dw(R, E, N, K, dy, x, off, dw, False, ws)
    assert c.coli_moe_get_status(ws) == c.COLI_ERR_BAD_INDEX
    assert torch.all(dw[1:4] == 7.0)
    _check(dw[4], dy[20:].double().T @ x[20:].double(), dy[20:].double().abs().T @ x[20:].double().abs(), 20)


def test_no_rows():
    from int4_routed_expert_coli_b200 import coli_moe as c
    E, N, K = 3, 16, 32
    e = torch.empty(0, K, dtype=torch.bfloat16, device="cuda")
    d = torch.empty(0, N, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(E, N, K, dtype=torch.bfloat16, device="cuda")
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    ws = c.grouped_workspace(0, E)
    c.coli_moe_grouped_mm(0, E, N, K, e, w, off, d, ws)
    c.coli_moe_grouped_mm_dx(0, E, N, K, d, w, off, e, ws)
    dw = torch.full((E, N, K), 7.0, device="cuda")
    c.coli_moe_grouped_mm_dw(0, E, N, K, d, e, off, dw, True, ws)
    assert torch.all(dw == 7.0)
    c.coli_moe_grouped_mm_dw(0, E, N, K, d, e, off, dw, False, ws)
    assert torch.all(dw == 0)
    # rows, but every group empty
    x = torch.ones(4, K, dtype=torch.bfloat16, device="cuda")
    dy = torch.ones(4, N, dtype=torch.bfloat16, device="cuda")
    out = torch.full((4, N), 7.0, device="cuda")
    c.coli_moe_grouped_mm(4, E, N, K, x, w, off, out, ws)
    assert torch.all(out == 7.0)
    dw.fill_(7.0)
    c.coli_moe_grouped_mm_dw(4, E, N, K, dy, x, off, dw, False, ws)
    assert torch.all(dw == 0)
    assert c.coli_moe_get_status(ws) == c.COLI_OK


def test_repeats_bit_for_bit_and_replays():
    """Cut tiles add their parts in a fixed order; captured calls replay on new
    inputs and new group sizes."""
    from int4_routed_expert_coli_b200 import coli_moe as c
    E, N, K = 8, 384, 2048
    counts = [1, 0, 9, 2, 0, 30, 1, 1]
    off, o = _offsets(counts)
    R = o[-1]
    g = _gen(6)
    x, w = _rn(g, R, K), _rn(g, E, N, K)
    ws = c.grouped_workspace(R, E)
    out = [torch.empty(R, N, device="cuda") for _ in range(5)]
    for t in out:
        c.coli_moe_grouped_mm(R, E, N, K, x, w, off, t, ws)
    for t in out[1:]:
        assert torch.equal(t, out[0])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        c.coli_moe_grouped_mm(R, E, N, K, x, w, off, out[1], ws)
    x.copy_(_rn(g, R, K))
    off.copy_(_offsets([0, 20, 0, 0, 22, 0, 0, 2])[0])
    graph.replay()
    c.coli_moe_grouped_mm(R, E, N, K, x, w, off, out[0], ws)
    assert torch.equal(out[0], out[1])
    assert c.coli_moe_get_status(ws) == c.COLI_OK


@pytest.mark.parametrize("offsets,kept", [
    ([0, 10, 5, 10, 30], [(0, 0, 10), (3, 10, 30)]),
    ([0, 20, 8, 30, 30, 40], [(0, 0, 20), (3, 30, 30), (4, 30, 40)]),
    # [40, 90) leaves the rows; [50, 90) would too; [3, 12) is free of earlier groups
    ([40, 90, 50, 90, 3, 12, 12, 2, 13, 20], [(4, 3, 12), (5, 12, 12), (8, 13, 20)]),
])
def test_groups_inside_an_earlier_one_are_skipped(offsets, kept):
    """No row belongs to two groups, whatever the offsets: one that starts inside
    an earlier group is left out like the pair that descends, and the same call
    gives the same bits."""
    from int4_routed_expert_coli_b200 import coli_moe as c
    E, R, N, K = len(offsets) - 1, 64, 264, 1040
    g = _gen(11)
    x, w, dy = _rn(g, R, K), _rn(g, E, N, K, scale=0.1), _rn(g, R, N)
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    ws = c.grouped_workspace(R, E)
    wq = w.to(torch.float8_e4m3fn)
    xq = torch.empty(R, K, dtype=torch.float8_e4m3fn, device="cuda")
    sx = torch.empty(-(-K // 128), R, device="cuda")
    c.coli_moe_fp8_quantize_rows(R, K, x, xq, sx)
    sw = torch.ones(E, -(-N // 128), -(-K // 128), device="cuda")
    X8 = xq.double() * sx.T.double().repeat_interleave(128, 1)[:, :K]
    for repeat in range(2):
        out, o8 = (torch.full((R, N), 7.0, device="cuda") for _ in range(2))
        dx, dw = torch.full((R, K), 7.0, device="cuda"), torch.full((E, N, K), 7.0, device="cuda")
        c.coli_moe_grouped_mm(R, E, N, K, x, w, off, out, ws)
        c.coli_moe_grouped_mm_dx(R, E, N, K, dy, w, off, dx, ws)
        c.coli_moe_grouped_mm_dw(R, E, N, K, dy, x, off, dw, False, ws)
        c.coli_moe_fp8_grouped_mm(R, E, N, K, xq, sx, wq, sw, off, o8, ws)
        assert c.coli_moe_get_status(ws) == c.COLI_ERR_BAD_INDEX
        if repeat:
            for a, b in zip(first, (out, dx, dw, o8)):
                assert torch.equal(a, b)
        first = out, dx, dw, o8
    free = torch.ones(R, dtype=torch.bool, device="cuda")
    for e, lo, hi in kept:
        free[lo:hi] = False
        X, W, D = x[lo:hi].double(), w[e].double(), dy[lo:hi].double()
        _check(out[lo:hi], X @ W.T, X.abs() @ W.abs().T, K)
        _check(dx[lo:hi], D @ W, D.abs() @ W.abs(), N)
        _check(dw[e], D.T @ X, D.abs().T @ X.abs(), hi - lo)
        W8 = wq[e].double()
        _check(o8[lo:hi], X8[lo:hi] @ W8.T, X8[lo:hi].abs() @ W8.abs().T, K)
    assert torch.all(out[free] == 7) and torch.all(dx[free] == 7) and torch.all(o8[free] == 7)
    skipped = [e for e in range(E) if e not in [k[0] for k in kept]]
    assert torch.all(dw[skipped] == 7)


def _poisoned(c, R, E):
    """A workspace whose partial sums are NaN until a call writes them."""
    ws = c.grouped_workspace(R, E)
    ws[c.COLI_WS_HEADER_BYTES:].fill_(255)
    return ws


def _has_parts(c, ws):
    return bool((ws[c.COLI_WS_HEADER_BYTES:] != 255).any())


# tiles cut between workers (asserted: partial sums in the workspace), in every
# direction: narrow tiles and pairs, several groups in one wave, ranges that start
# and end inside a group or hold several groups, sizes that are no multiple of the
# K-block or the MMA step
CUT = [
    ("mm", [1] * 8, 512, 6144),
    ("mm", [3, 0, 40, 1], 264, 8200),
    ("mm", [513], 2312, 6144),
    ("dx", [8], 4096, 6144),
    ("dx", [3, 0, 2, 3], 4104, 520),
    ("dx", [513], 6144, 2312),
    ("dw", [16371], 512, 512),
    ("dw", [0, 9003, 0, 37, 7000, 0], 512, 520),
    ("dw", [5000, 5001, 4999], 136, 264),
]


@pytest.mark.parametrize("out_dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("op,counts,N,K", CUT)
def test_cut_tiles(op, counts, N, K, out_dt):
    from int4_routed_expert_coli_b200 import coli_moe as c
    E = len(counts)
    first, behind = 3, 5
    off, o = _offsets(counts, first)
    R = o[-1] + behind
    g = _gen(N * 41 + K)
    x, dy = _rn(g, R, K), _rn(g, R, N)
    w = _rn(g, E, N, K, scale=0.1) if op != "dw" else None
    for t in (x, dy):
        t[:first] = NAN
        t[o[-1]:] = float("inf")
    shape = {"mm": (R, N), "dx": (R, K), "dw": (E, N, K)}[op]
    outs = []
    for _ in range(4):
        out, ws = torch.full(shape, NAN, dtype=out_dt, device="cuda"), _poisoned(c, R, E)
        if op == "mm":
            c.coli_moe_grouped_mm(R, E, N, K, x, w, off, out, ws)
        elif op == "dx":
            c.coli_moe_grouped_mm_dx(R, E, N, K, dy, w, off, out, ws)
        else:
            c.coli_moe_grouped_mm_dw(R, E, N, K, dy, x, off, out, False, ws)
        assert c.coli_moe_get_status(ws) == c.COLI_OK and _has_parts(c, ws)
        outs.append(out)
    for t in outs[1:]:       # added in a fixed order, whoever finishes last
        assert torch.equal(t.view(torch.uint8), outs[0].view(torch.uint8))
    for e in range(E):
        lo, hi = o[e], o[e + 1]
        X, D = x[lo:hi].double(), dy[lo:hi].double()
        if op == "dw":
            _check(outs[0][e], D.T @ X, D.abs().T @ X.abs(), hi - lo)
            continue
        W = w[e].double()
        if op == "mm":
            _check(outs[0][lo:hi], X @ W.T, X.abs() @ W.abs().T, K)
        else:
            _check(outs[0][lo:hi], D @ W, D.abs() @ W.abs(), N)
    if op != "dw":
        assert torch.isnan(outs[0][:first]).all() and torch.isnan(outs[0][o[-1]:]).all()


@pytest.mark.parametrize("out_dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("counts,N,K", [([1] * 8, 512, 6144), ([513], 2312, 6144)])
def test_fp8_cut_tiles(counts, N, K, out_dt):
    from int4_routed_expert_coli_b200 import coli_moe as c
    E = len(counts)
    off, o = _offsets(counts)
    R, nb, kb = o[-1], -(-N // 128), -(-K // 128)
    g = _gen(N * 43 + K)
    x = _rn(g, R, K)
    wq = _rn(g, E, N, K, dt=torch.float32, scale=100.0).clamp(-448, 448).to(torch.float8_e4m3fn)
    sw = torch.rand(E, nb, kb, generator=g, device="cuda") * 1e-3 + 1e-4
    xq = torch.empty(R, K, dtype=torch.float8_e4m3fn, device="cuda")
    sx = torch.empty(kb, R, device="cuda")
    c.coli_moe_fp8_quantize_rows(R, K, x, xq, sx)
    outs = []
    for _ in range(4):
        out, ws = torch.full((R, N), NAN, dtype=out_dt, device="cuda"), _poisoned(c, R, E)
        c.coli_moe_fp8_grouped_mm(R, E, N, K, xq, sx, wq, sw, off, out, ws)
        assert c.coli_moe_get_status(ws) == c.COLI_OK and _has_parts(c, ws)
        outs.append(out)
    for t in outs[1:]:
        assert torch.equal(t, outs[0])
    X = xq.double() * sx.T.double().repeat_interleave(128, 1)[:, :K]
    for e in range(E):
        lo, hi = o[e], o[e + 1]
        W = wq[e].double() * sw[e].double().repeat_interleave(128, 0)[:N] \
            .repeat_interleave(128, 1)[:, :K]
        _check(outs[0][lo:hi], X[lo:hi] @ W.T, X[lo:hi].abs() @ W.abs().T, K)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("counts,N,K", [([16371], 512, 512), ([0, 9003, 0, 37, 7000], 264, 520)])
def test_cut_weight_gradient_accumulates(counts, N, K, dt):
    from int4_routed_expert_coli_b200 import coli_moe as c
    off, o = _offsets(counts)
    R, E = o[-1], len(counts)
    g = _gen(12)
    x, dy, dw = _rn(g, R, K), _rn(g, R, N), _rn(g, E, N, K, dt=dt)
    old, ws = dw.double(), _poisoned(c, R, E)
    c.coli_moe_grouped_mm_dw(R, E, N, K, dy, x, off, dw, True, ws)
    assert c.coli_moe_get_status(ws) == c.COLI_OK and _has_parts(c, ws)
    for e in range(E):
        if counts[e] == 0:
            assert torch.equal(dw[e].double(), old[e])
            continue
        X, D = x[o[e]:o[e + 1]].double(), dy[o[e]:o[e + 1]].double()
        _check(dw[e], old[e] + D.T @ X, old[e].abs() + D.abs().T @ X.abs(), counts[e])


@pytest.mark.parametrize("op,counts,N,K", [("mm", [64], 136, 16384), ("mm", [600], 2312, 16384),
                                           ("dx", [64], 16384, 136), ("dx", [600], 16384, 2312),
                                           ("dw", [16384], 264, 520)])
def test_long_sums_leave_the_tensor_cores_in_chains(op, counts, N, K):
    """Sums of 16384 positive products.  A chain of at most 768 products is 48
    truncating additions of 16, each at most 2^-23 of the chain's sum; the 22 chains
    (and up to 16 ranges of a cut tile) are added in fp32, each at most 2^-24 of the
    whole: (48 + 19) 2^-23.  One chain of 16384, 1024 truncations of about half a
    step of a sum that grows from nothing, is about 2e-5 off: more than twice that."""
    from int4_routed_expert_coli_b200 import coli_moe as c
    g = _gen(13)
    R, E = counts[0], 1

    def pos(*shape):
        return (torch.rand(*shape, generator=g, device="cuda") + 0.5).bfloat16()
    off, ws = _offsets(counts)[0], c.grouped_workspace(R, E)
    x, dy, w = pos(R, K), pos(R, N), pos(E, N, K)
    if op == "mm":
        out, ref = torch.empty(R, N, device="cuda"), x.double() @ w[0].double().T
        c.coli_moe_grouped_mm(R, E, N, K, x, w, off, out, ws)
    elif op == "dx":
        out, ref = torch.empty(R, K, device="cuda"), dy.double() @ w[0].double()
        c.coli_moe_grouped_mm_dx(R, E, N, K, dy, w, off, out, ws)
    else:
        out, ref = torch.empty(E, N, K, device="cuda"), (dy.double().T @ x.double())[None]
        c.coli_moe_grouped_mm_dw(R, E, N, K, dy, x, off, out, False, ws)
    assert c.coli_moe_get_status(ws) == c.COLI_OK
    assert float(((out.double() - ref).abs() / ref).max()) <= 67 * 2.0 ** -23
