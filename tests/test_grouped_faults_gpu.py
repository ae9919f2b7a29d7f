"""The grouped products' bounded waits, without faulting the GPU: a stage that
is never filled makes the waits of every role run out; the kernel ends, the
status word reads COLI_ERR_TIMEOUT, and after a clear the same call gives the
same bits as before."""
import pytest
import torch

from gpu_util import requires_gpu

pytestmark = [pytest.mark.gpu, requires_gpu]


def _rn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").bfloat16()


def _call(c, op, counts, N, K, ws, seed=0):
    """One call of `op`; returns a function that makes it into a new output."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    E, R = len(counts), sum(counts)
    off = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32,
                       device="cuda")
    x, dy, w = _rn(g, R, K), _rn(g, R, N), _rn(g, E, N, K)

    def run():
        shape = {"mm": (R, N), "fp8": (R, N), "dx": (R, K), "dw": (E, N, K)}[op]
        out = torch.zeros(shape, device="cuda")
        if op == "mm":
            c.coli_moe_grouped_mm(R, E, N, K, x, w, off, out, ws)
        elif op == "dx":
            c.coli_moe_grouped_mm_dx(R, E, N, K, dy, w, off, out, ws)
        elif op == "dw":
            c.coli_moe_grouped_mm_dw(R, E, N, K, dy, x, off, out, False, ws)
        else:
            kb = -(-K // 128)
            xq = torch.empty(R, K, dtype=torch.float8_e4m3fn, device="cuda")
            xs = torch.empty(kb, R, device="cuda")
            c.coli_moe_fp8_quantize_rows(R, K, x, xq, xs)
            wq = w.to(torch.float8_e4m3fn)
            sw = torch.full((E, -(-N // 128), kb), 0.25, device="cuda")
            c.coli_moe_fp8_grouped_mm(R, E, N, K, xq, xs, wq, sw, off, out, ws)
        return out
    return run


# narrow and wide tiles, whole and cut (a cut tile's partial sums are added by
# whoever finishes last), one CTA and pairs, e4m3 with the weights and the rows as M
@pytest.mark.parametrize("op,counts,N,K", [
    ("mm", [1] * 8 + [0] * 24, 512, 4096),
    ("mm", [3000], 520, 200),
    ("mm", [513], 2312, 6144),
    ("dx", [8], 4096, 6144),
    ("dw", [37, 3, 60], 128, 192),
    ("dw", [16371], 512, 512),
    ("fp8", [1] * 8, 512, 6144),
    ("fp8", [513], 2312, 6144),
])
def test_withheld_stage_times_out_and_the_next_call_is_right(op, counts, N, K):
    from int4_routed_expert_coli_b200 import coli_moe as c
    ws = c.grouped_workspace(sum(counts), len(counts))
    run = _call(c, op, counts, N, K, ws)
    want = run()
    assert c.coli_moe_get_status(ws) == c.COLI_OK
    assert c.coli_moe_debug_inject(c.COLI_INJECT_WITHHOLD_GROUPED) == c.COLI_OK
    try:
        run()
    finally:
        c.coli_moe_debug_inject(0)
    assert c.coli_moe_get_status(ws) == c.COLI_ERR_TIMEOUT
    c.coli_moe_workspace_clear(ws)
    got = run()
    assert c.coli_moe_get_status(ws) == c.COLI_OK
    assert torch.equal(got, want)


@pytest.mark.parametrize("op,counts,N,K", [("mm", [700], 2312, 6144), ("dw", [3000, 37], 512, 512),
                                           ("fp8", [700], 2312, 6144)])
def test_a_call_that_gave_up_leaves_the_next_one_alone(op, counts, N, K):
    """Its copies and MMAs in flight end with it: calls that follow at once, on a
    workspace of their own, start on its SMs and are right."""
    from int4_routed_expert_coli_b200 import coli_moe as c
    R, E = sum(counts), len(counts)
    bad, ws = c.grouped_workspace(R, E), c.grouped_workspace(R, E)
    first, run = _call(c, op, counts, N, K, bad, seed=1), _call(c, op, counts, N, K, ws)
    want = run()
    torch.cuda.synchronize()
    assert c.coli_moe_debug_inject(c.COLI_INJECT_SHORT_WAITS) == c.COLI_OK
    assert c.coli_moe_debug_inject(c.COLI_INJECT_WITHHOLD_GROUPED) == c.COLI_OK
    try:
        first()
    finally:
        c.coli_moe_debug_inject(0)
    got = [run() for _ in range(4)]
    assert c.coli_moe_get_status(bad) == c.COLI_ERR_TIMEOUT
    assert c.coli_moe_get_status(ws) == c.COLI_OK
    for t in got:
        assert torch.equal(t, want)


def test_work_longer_than_a_wait_is_no_timeout():
    """A weight gradient whose first group, of whole K-blocks, takes several times
    a wait's limit (2.6e5 rows of 8192 x 8192, about 25 ms, waits of 5 ms) before
    the group whose last K-block is cut."""
    from int4_routed_expert_coli_b200 import coli_moe as c
    counts, N, K = [1 << 18, 37], 8192, 8192
    R, E = sum(counts), 2
    g = torch.Generator(device="cuda").manual_seed(3)
    x, dy = (torch.empty(R, 8192, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
             for _ in range(2))
    off = torch.tensor([0, counts[0], R], dtype=torch.int32, device="cuda")
    ws = c.grouped_workspace(R, E)
    dw = [torch.zeros(E, N, K, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    c.coli_moe_grouped_mm_dw(R, E, N, K, dy, x, off, dw[0], False, ws)
    assert c.coli_moe_get_status(ws) == c.COLI_OK
    assert c.coli_moe_debug_inject(c.COLI_INJECT_SHORT_WAITS) == c.COLI_OK
    try:
        c.coli_moe_grouped_mm_dw(R, E, N, K, dy, x, off, dw[1], False, ws)
    finally:
        c.coli_moe_debug_inject(0)
    assert c.coli_moe_get_status(ws) == c.COLI_OK
    assert torch.equal(dw[0], dw[1])
    rows, cols = slice(N - 8, N), slice(K - 8, K)
    for e, r in ((0, slice(0, counts[0])), (1, slice(counts[0], R))):
        ref = dy[r, rows].double().T @ x[r, cols].double()
        mag = dy[r, rows].double().abs().T @ x[r, cols].double().abs()
        tol = 2.0 ** -8 * ref.abs() + (counts[e] / 16 + 64) * 2.0 ** -23 * mag
        assert torch.all((dw[0][e, rows, cols].double() - ref).abs() <= tol)
