"""The norms, the grouped products and the 8-bit product as a block uses them
together with the routing, the batch-union and the combine, forward and
backward; calls on several streams, a shared workspace, arrays past 32-bit
offsets, and what the binding refuses."""
import pytest
import torch

from gpu_util import requires_gpu
from int4_routed_expert_coli_b200 import synth

pytestmark = [pytest.mark.gpu, requires_gpu]

EPS = 1e-5


def _rn(g, *shape, dt=torch.bfloat16, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dt)


def _rel(got, ref):
    return float((got.double() - ref).norm() / ref.norm())


def _routed(c, logits, k):
    """Routing, union lists and each list entry's token and gate weight."""
    T, E = logits.shape
    i32 = dict(dtype=torch.int32, device="cuda")
    idx, w = torch.empty(T, k, **i32), torch.empty(T, k, device="cuda")
    c.coli_moe_route(T, E, k, logits, idx, w)
    counts, offsets, pairs = torch.empty(E, **i32), torch.empty(E + 1, **i32), torch.empty(T * k, **i32)
    active, na = torch.empty(E, **i32), torch.empty(1, **i32)
    c.coli_moe_union(T, E, k, idx, counts, offsets, pairs, active, na)
    return idx, w, offsets, pairs.long()


class Block:
    """One pre- and post-normed block of bf16 experts around the library."""

    def __init__(self, T, H, I, E, k, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.T, self.H, self.I, self.E, self.k = T, H, I, E, k
        self.x = _rn(g, T, H, scale=2.0)
        self.pre_w, self.post_w = 1 + 0.2 * _rn(g, H, dt=torch.float32), 1 + 0.2 * _rn(g, H, dt=torch.float32)
        self.w1, self.w2 = _rn(g, E, 2 * I, H, scale=H ** -0.5), _rn(g, E, H, I, scale=I ** -0.5)
        self.logits = torch.randn(T, E, generator=g, device="cuda")
        self.alpha = 0.8
        self.grad = _rn(g, T, H)

    def reference(self, idx, w):
        """Output and gradients in 64 bits, routing given."""
        d = torch.float64
        leaf = {n: getattr(self, n).to(d).requires_grad_(True)
                for n in ("x", "pre_w", "post_w", "w1", "w2")}
        x = leaf["x"]
        o = x / torch.sqrt((x * x).mean(1, keepdim=True) + EPS) * leaf["pre_w"]
        y = torch.zeros_like(o)
        for e in range(self.E):
            t, j = torch.nonzero(idx == e, as_tuple=True)
            if t.numel() == 0:
                continue
            gu = o[t] @ leaf["w1"][e].T
            h = torch.nn.functional.silu(gu[:, :self.I]) * gu[:, self.I:]
            y = y.index_add(0, t, (h @ leaf["w2"][e].T) * w[t, j].to(d)[:, None])
        n = y / torch.sqrt((y * y).mean(1, keepdim=True) + EPS) * leaf["post_w"]
        s = x + self.alpha * n
        s.backward(self.grad.to(d))
        return s.detach(), {n: v.grad for n, v in leaf.items()}


@pytest.mark.parametrize("T,H,I,E,k", [(1, 256, 128, 16, 2), (40, 256, 128, 16, 2),
                                       (333, 512, 264, 12, 3)])
def test_block_forward_and_backward(T, H, I, E, k):
    """Every stage rounds once to bf16, at most half a step (2^-8) of each value.
    Four stages lead to the output and the residual sum adds an exact x; the
    gradients pass at most nine (four forward, five back).  A stage's error is
    carried on by products and norms that keep its share of the whole, so each
    result is within its number of stages times 2^-8 in the 2-norm."""
    from int4_routed_expert_coli_b200 import coli_moe as c
    b = Block(T, H, I, E, k, seed=T + H)
    P, dev = T * k, "cuda"
    bf = dict(dtype=torch.bfloat16, device=dev)
    ws = c.grouped_workspace(P, E)
    # forward
    o = torch.empty(T, H, **bf)
    c.coli_moe_block_norm(T, H, b.x, None, None, None, c.COLI_GATE_NONE, 1.0, b.pre_w, EPS, None, o)
    idx, w, off, pairs = _routed(c, b.logits, k)
    tok, gw = pairs // k, w.view(-1)[pairs]
    xg = o[tok].contiguous()
    gu, yr = torch.empty(P, 2 * I, **bf), torch.empty(P, H, device=dev)
    c.coli_moe_grouped_mm(P, E, 2 * I, H, xg, b.w1, off, gu, ws)
    gf, uf = gu.float().split(I, 1)
    h = (torch.nn.functional.silu(gf) * uf).bfloat16()
    c.coli_moe_grouped_mm(P, E, H, I, h, b.w2, off, yr, ws)
    rows = torch.empty(P, H, device=dev)
    rows[pairs] = yr * gw[:, None]
    y, s = torch.empty(T, H, **bf), torch.empty(T, H, **bf)
    c.coli_moe_combine_rows(T, k, H, rows, None, None, y, c.COLI_OUT_BF16)
    c.coli_moe_block_norm(T, H, b.x, y, b.post_w, None, c.COLI_GATE_NONE, b.alpha, None, EPS, s, None)
    ref, want = b.reference(idx.long(), w)
    assert c.coli_moe_get_status(ws) == c.COLI_OK
    assert _rel(s, ref) <= 5 * 2.0 ** -8

    # backward
    nws = torch.empty(c.coli_moe_block_norm_workspace_size(T, H), dtype=torch.uint8, device=dev)
    dx, dy = torch.empty(T, H, **bf), torch.empty(T, H, **bf)
    dpost = torch.empty(H, device=dev)
    c.coli_moe_block_norm_backward(T, H, None, b.grad, None, y, b.post_w, None, c.COLI_GATE_NONE,
                                   b.alpha, None, EPS, dx, dy, None, dpost, None, nws)
    dyr = (dy.float()[tok] * gw[:, None]).bfloat16()
    dw2, dw1 = torch.empty(E, H, I, device=dev), torch.empty(E, 2 * I, H, device=dev)
    dh = torch.empty(P, I, device=dev)
    c.coli_moe_grouped_mm_dx(P, E, H, I, dyr, b.w2, off, dh, ws)
    c.coli_moe_grouped_mm_dw(P, E, H, I, dyr, h, off, dw2, False, ws)
    sg = torch.sigmoid(gf)
    dgu = torch.cat([dh * uf * (sg + gf * sg * (1 - sg)), dh * gf * sg], 1).bfloat16()
    dxg = torch.empty(P, H, device=dev)
    c.coli_moe_grouped_mm_dx(P, E, 2 * I, H, dgu, b.w1, off, dxg, ws)
    c.coli_moe_grouped_mm_dw(P, E, 2 * I, H, dgu, xg, off, dw1, False, ws)
    do = torch.zeros(T, H, device=dev).index_add_(0, tok, dxg).bfloat16()
    dpre = torch.empty(H, device=dev)
    c.coli_moe_block_norm_backward(T, H, do, dx, b.x, None, None, None, c.COLI_GATE_NONE, 1.0,
                                   b.pre_w, EPS, dx, None, dpre, None, None, nws)
    assert c.coli_moe_get_status(ws) == c.COLI_OK
    for name, got in (("post_w", dpost), ("w2", dw2), ("w1", dw1), ("pre_w", dpre), ("x", dx)):
        assert _rel(got, want[name]) <= 9 * 2.0 ** -8, (name, _rel(got, want[name]))


@pytest.mark.parametrize("T", [1, 50, 400])
def test_experts_in_8_bits(T):
    """The block's experts in e4m3: the products of the quantised rows are those
    of a bf16 block within the two quantisations, half a step of e4m3 (2^-4) of
    each value, one behind the other: 2 * 2^-4 in the 2-norm; against the same
    quantised values in 64 bits, only the output's bf16 rounding is left."""
    from int4_routed_expert_coli_b200 import coli_moe as c
    H, I, E, k = 512, 256, 8, 2
    b = Block(T, H, I, E, k, seed=T)
    P = T * k
    idx, w, off, pairs = _routed(c, b.logits, k)
    x = b.x[pairs // k].contiguous()

    def weights(t):
        n, m = t.shape[1] // 128, t.shape[2] // 128
        v = t.float().view(E, n, 128, m, 128)
        s = v.abs().amax((2, 4)) / 448.0
        q = (v / s[:, :, None, :, None]).to(torch.float8_e4m3fn)
        deq = (q.double() * s.double()[:, :, None, :, None]).view(t.shape)
        return q.view(t.shape).contiguous(), s.contiguous(), deq

    def product(v, wt, out):
        R, K = v.shape
        q = torch.empty(R, K, dtype=torch.float8_e4m3fn, device="cuda")
        s = torch.empty(K // 128, R, device="cuda")
        c.coli_moe_fp8_quantize_rows(R, K, v, q, s)
        c.coli_moe_fp8_grouped_mm(R, E, out.shape[1], K, q, s, wt[0], wt[1], off, out, ws)
        return q.double() * s.T.double().repeat_interleave(128, 1)

    ws = c.grouped_workspace(P, E)
    w1, w2 = weights(b.w1), weights(b.w2)
    gu = torch.empty(P, 2 * I, device="cuda", dtype=torch.bfloat16)
    y = torch.empty(P, H, device="cuda", dtype=torch.bfloat16)
    xq = product(x, w1, gu)
    h = (torch.nn.functional.silu(gu.float()[:, :I]) * gu.float()[:, I:]).bfloat16()
    hq = product(h, w2, y)
    assert c.coli_moe_get_status(ws) == c.COLI_OK
    o = off.tolist()
    y8, y16 = torch.empty(P, H, dtype=torch.float64, device="cuda"), torch.empty(
        P, H, dtype=torch.float64, device="cuda")
    gu8 = torch.empty(P, 2 * I, dtype=torch.float64, device="cuda")
    for e in range(E):
        r = slice(o[e], o[e + 1])
        gu8[r] = xq[r] @ w1[2][e].T
        y8[r] = hq[r] @ w2[2][e].T
        g, u = (x[r].double() @ w1[2][e].T).split(I, 1)
        y16[r] = (torch.nn.functional.silu(g) * u) @ w2[2][e].T
    assert _rel(gu, gu8) <= 2.0 ** -8 and _rel(y, y8) <= 2.0 ** -8
    assert _rel(y, y16) <= 2 * 2.0 ** -4


def test_two_streams_at_once():
    """Calls on two streams, each with its own workspace, and on a stream that is
    not the current one."""
    from int4_routed_expert_coli_b200 import coli_moe as c
    g = torch.Generator(device="cuda").manual_seed(1)
    E, N, K, R = 4, 512, 2048, 150
    x, w = [_rn(g, R, K) for _ in range(2)], _rn(g, E, N, K)
    off = torch.tensor([0, 20, 21, 100, R], dtype=torch.int32, device="cuda")
    ws = [c.grouped_workspace(R, E) for _ in range(2)]
    want = [torch.empty(R, N, device="cuda") for _ in range(2)]
    for i in range(2):
        c.coli_moe_grouped_mm(R, E, N, K, x[i], w, off, want[i], ws[i])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[torch.empty(R, N, device="cuda") for _ in range(2)] for _ in range(8)]
    torch.cuda.synchronize()
    for n in range(8):
        for i in range(2):
            c.coli_moe_grouped_mm(R, E, N, K, x[i], w, off, got[n][i], ws[i], stream=streams[i])
    torch.cuda.synchronize()
    for n in range(8):
        for i in range(2):
            assert torch.equal(got[n][i], want[i])
    with torch.cuda.stream(streams[0]):
        c.coli_moe_grouped_mm(R, E, N, K, x[0], w, off, got[0][1], ws[0])
    streams[0].synchronize()
    assert torch.equal(got[0][1], want[0])


def test_workspace_shared_with_the_layer():
    """One workspace, in stream order, for the layer step and a grouped product:
    each leaves it as the other needs it."""
    from int4_routed_expert_coli_b200 import coli_moe as c
    H, I, E, k, T = 256, 128, 16, 2, 4
    bank = synth.make_expert_bank(H, I, E + 1, seed=0, device="cuda")
    layer = c.MoELayer(bank, n_routed=E, top_k=k, n_shared=1)
    x = synth.make_activations(T, H, seed=0, device="cuda")
    lg = synth.make_logits_normal(T, E, seed=1, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(2)
    R, N, K = 9, 384, 4096
    xr, w = _rn(g, R, K), _rn(g, E, N, K)
    off = torch.tensor([0] * 8 + [R] * 9, dtype=torch.int32, device="cuda")
    n = max(layer.workspace_size(T), c.coli_moe_grouped_workspace_size(R, E))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    c.coli_moe_workspace_clear(ws)
    outs, prods = [], []
    for _ in range(3):
        outs.append(layer.layer(x, logits=lg, ws=ws))
        p = torch.empty(R, N, device="cuda")
        c.coli_moe_grouped_mm(R, E, N, K, xr, w, off, p, ws)
        prods.append(p)
    assert c.coli_moe_get_status(ws) == c.COLI_OK
    for a in (outs, prods):
        assert torch.equal(a[0], a[1]) and torch.equal(a[0], a[2])


def test_offsets_past_32_bits():
    """Arrays of more than 2^31 elements, checked at their ends."""
    from int4_routed_expert_coli_b200 import coli_moe as c
    g = torch.Generator(device="cuda").manual_seed(3)
    # weights: 3 x 32768 x 32768 elements; one row each to the first and last expert
    E, N, K = 3, 32768, 32768
    w = torch.zeros(E, N, K, dtype=torch.bfloat16, device="cuda")
    w[0, :64], w[2, -64:] = _rn(g, 64, K), _rn(g, 64, K)
    x = _rn(g, 2, K)
    off = torch.tensor([0, 1, 1, 2], dtype=torch.int32, device="cuda")
    out = torch.empty(2, N, device="cuda")
    ws = c.grouped_workspace(2, E)
    c.coli_moe_grouped_mm(2, E, N, K, x, w, off, out, ws)
    for r, e, rows in ((0, 0, slice(0, 64)), (1, 2, slice(N - 64, N))):
        ref = w[e, rows].double() @ x[r].double()
        mag = w[e, rows].double().abs() @ x[r].double().abs()
        assert torch.all((out[r, rows].double() - ref).abs() <= (K / 16 + 64) * 2.0 ** -23 * mag)
    dw = w  # the gradient of the last expert, over the weights
    dy = _rn(g, 2, N)
    c.coli_moe_grouped_mm_dw(2, E, N, K, dy, x, off, dw, False, ws)
    ref = dy[1, -8:].double()[:, None] * x[1, -8:].double()[None, :]
    assert torch.all((dw[2, -8:, -8:].double() - ref).abs() <= 2.0 ** -8 * ref.abs())
    assert torch.all(dw[1] == 0)
    del w, dw, out
    # rows: 140000 x 16384
    T, H = 140000, 16384
    x = torch.ones(T, H, dtype=torch.bfloat16, device="cuda")
    x[-1] = _rn(g, H)
    o = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    pre = torch.ones(H, device="cuda")
    c.coli_moe_block_norm(T, H, x, None, None, None, c.COLI_GATE_NONE, 1.0, pre, EPS, None, o)
    v = x[-1].double()
    ref = v / torch.sqrt((v * v).mean() + EPS)
    assert torch.all((o[-1].double() - ref).abs() <= (2.0 ** -8 + 2.0 ** -16) * ref.abs())
    q = torch.empty(T, H, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty(H // 128, T, device="cuda")
    c.coli_moe_fp8_quantize_rows(T, H, x, q, s)
    top = x[-1].float().view(-1, 128).abs().amax(1) / 448.0
    assert torch.all((s[:, -1] - top).abs() <= 2.0 ** -23 * top)


def test_binding_checks_sizes_types_and_layout():
    from int4_routed_expert_coli_b200 import coli_moe as c
    T, H = 4, 64
    x, w = torch.zeros(T, H, device="cuda"), torch.ones(H, device="cuda")

    def norm(**kw):
        a = dict(x=x, y=None, post_w=None, gate=None, kind=c.COLI_GATE_NONE, pre_w=w,
                 s=torch.empty_like(x), o=torch.empty_like(x))
        a.update(kw)
        c.coli_moe_block_norm(T, H, a["x"], a["y"], a["post_w"], a["gate"], a["kind"], 1.0,
                              a["pre_w"], EPS, a["s"], a["o"])

    norm()
    for kw in (dict(x=x[:3]), dict(x=x.half()), dict(x=x.T.contiguous().T), dict(pre_w=w[:63]),
               dict(pre_w=w.bfloat16()), dict(s=x.bfloat16()), dict(y=x[:, :32].contiguous()),
               dict(gate=w[:3], kind=c.COLI_GATE_TOKEN), dict(x=x.cpu())):
        with pytest.raises(ValueError):
            norm(**kw)
    with pytest.raises(c.ColiError):
        norm(pre_w=None)
    with pytest.raises(TypeError):
        norm(pre_w=3.0)

    R, E, N, K = 3, 2, 64, 128
    xb, wb = torch.zeros(R, K, device="cuda", dtype=torch.bfloat16), torch.zeros(
        E, N, K, device="cuda", dtype=torch.bfloat16)
    off = torch.tensor([0, 1, 3], dtype=torch.int32, device="cuda")
    out, ws = torch.empty(R, N, device="cuda"), c.grouped_workspace(R, E)
    c.coli_moe_grouped_mm(R, E, N, K, xb, wb, off, out, ws)
    for bad in ((xb[:2], wb, off, out), (xb, wb[:1], off, out), (xb, wb, off[:2], out),
                (xb, wb, off.long(), out), (xb.float(), wb, off, out), (xb, wb, off, out[:, :32])):
        with pytest.raises(ValueError):
            c.coli_moe_grouped_mm(R, E, N, K, *bad, ws)
    with pytest.raises(c.ColiError):
        c.coli_moe_grouped_mm(R, E, N, K, xb, wb, off, out, ws[:c.COLI_WS_HEADER_BYTES])
    assert c.coli_moe_grouped_mm(R, E, 60, K, xb, torch.zeros(E, 60, K, device="cuda",
                                 dtype=torch.bfloat16), off, torch.empty(R, 60, device="cuda"), ws,
                                 raise_on_error=False) == c.COLI_ERR_SHAPE


def test_two_graphs_share_a_workspace():
    """Captured one after the other with one workspace (cut tiles' partial sums,
    counters, column sums), replayed in turn: the bits of the eager calls."""
    from int4_routed_expert_coli_b200 import coli_moe as c
    R, E, N, K = 9, 4, 264, 2048
    g = torch.Generator(device="cuda").manual_seed(21)
    x, w, dy = (torch.randn(*s, generator=g, device="cuda").bfloat16()
                for s in ((R, K), (E, N, K), (R, N)))
    off = torch.tensor([0, 1, 5, 5, R], dtype=torch.int32, device="cuda")
    ws = c.grouped_workspace(R, E)
    out, dw = torch.empty(R, N, device="cuda"), torch.empty(E, N, K, device="cuda")

    def forward():
        c.coli_moe_grouped_mm(R, E, N, K, x, w, off, out, ws)

    def backward():
        c.coli_moe_grouped_mm_dw(R, E, N, K, dy, x, off, dw, False, ws)

    forward(), backward()
    want = out.clone(), dw.clone()
    torch.cuda.synchronize()
    graphs = []
    for f in (forward, backward):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            f()
    for i in (0, 1, 1, 0, 0, 1):
        (out, dw)[i].fill_(float("nan"))
        graphs[i].replay()
        assert torch.equal((out, dw)[i], want[i])
    assert c.coli_moe_get_status(ws) == c.COLI_OK


def test_two_host_threads():
    """Calls from two threads on two streams, of kernels and widths that need
    different amounts of shared memory."""
    import threading

    from int4_routed_expert_coli_b200 import coli_moe as c
    errors = []

    def work(H, seed):
        try:
            T = 700
            with torch.cuda.stream(torch.cuda.Stream()):
                g = torch.Generator(device="cuda").manual_seed(seed)
                x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
                pre = torch.ones(H, device="cuda")
                o, want = torch.empty_like(x), None
                for _ in range(100):
                    c.coli_moe_block_norm(T, H, x, None, None, None, c.COLI_GATE_NONE, 1.0, pre,
                                          1e-5, None, o)
                    if want is None:
                        want = o.clone()
                    c.coli_moe_block_norm(T, H, x, x, None, None, c.COLI_GATE_NONE, 0.0, pre, 1e-5,
                                          None, o)
                    assert torch.equal(o, want)
        except BaseException as e:  # noqa: BLE001 - handed to the test's own thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(H, i)) for i, H in enumerate((2048, 6144, 8192))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


def test_two_streams_and_graphs_with_cut_tiles():
    """Products whose tiles are cut (partial sums in the workspace), the weight
    gradient and the backward norm: on two streams at once, each with workspaces of
    its own, and captured into two graphs that share workspaces, replayed in turn:
    the bits of the eager calls."""
    from int4_routed_expert_coli_b200 import coli_moe as c
    g = torch.Generator(device="cuda").manual_seed(31)
    E, N, K, counts = 4, 264, 6144, [1, 4, 0, 4]
    R, T, H = sum(counts), 300, 776
    x, w, dy = _rn(g, R, K), _rn(g, E, N, K), _rn(g, R, N)
    off = torch.tensor([0, 1, 5, 5, 9], dtype=torch.int32, device="cuda")
    R2, n2 = 9003, 136
    x2, dy2 = _rn(g, R2, n2), _rn(g, R2, n2)
    off2 = torch.tensor([0, R2], dtype=torch.int32, device="cuda")
    s, y, do = _rn(g, T, H), _rn(g, T, H), _rn(g, T, H)
    pw, qw = torch.ones(H, device="cuda"), torch.ones(H, device="cuda")

    class Set:
        def __init__(self):
            self.ws = c.grouped_workspace(R2, E)
            self.ws[c.COLI_WS_HEADER_BYTES:].fill_(255)
            self.nws = torch.empty(c.coli_moe_block_norm_workspace_size(T, H), dtype=torch.uint8,
                                   device="cuda")
            self.res = [torch.empty(R, N, device="cuda"), torch.empty(1, n2, n2, device="cuda"),
                        torch.empty_like(s), torch.empty_like(y), torch.empty_like(pw),
                        torch.empty_like(qw)]

        def products(self):
            c.coli_moe_grouped_mm(R, E, N, K, x, w, off, self.res[0], self.ws)
            c.coli_moe_grouped_mm_dw(R2, 1, n2, n2, dy2, x2, off2, self.res[1], False, self.ws)

        def norm(self):
            c.coli_moe_block_norm_backward(T, H, do, None, s, y, pw, None, c.COLI_GATE_NONE, 0.5, qw,
                                           EPS, self.res[2], self.res[3], self.res[4], self.res[5],
                                           None, self.nws)

        def wipe(self):
            for t in self.res:
                t.fill_(float("nan"))

    a, b = Set(), Set()
    a.products(), a.norm()
    assert (a.ws[c.COLI_WS_HEADER_BYTES:] != 255).any()
    want = [t.clone() for t in a.res]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(6):
        a.wipe(), b.wipe()
        torch.cuda.synchronize()
        for st, v in zip(streams, (a, b)):
            with torch.cuda.stream(st):
                v.products(), v.norm(), v.products()
        torch.cuda.synchronize()
        for v in (a, b):
            assert all(torch.equal(t, u) for t, u in zip(v.res, want))
    graphs = []
    for f in (lambda: (a.products(), a.norm()), lambda: (a.norm(), a.products())):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            f()
    for i in (0, 1, 1, 0, 0, 1):
        a.wipe()
        graphs[i].replay()
        assert all(torch.equal(t, u) for t, u in zip(a.res, want))
    for v in (a, b):
        assert c.coli_moe_get_status(v.ws) == c.COLI_OK
