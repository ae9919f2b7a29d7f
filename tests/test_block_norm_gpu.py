"""Block norms (coli_moe_block_norm and its backward) against the formulas in
64 bits, and the gradients against differences.

Tolerances, u = 2^-24 (half a step of fp32).  A row's mean of squares sums up
to 64 positive terms per thread and 10 butterfly levels: at most 74 u off,
halved by the root, plus 2 ulp of rsqrtf: an inverse RMS is within 41 u; with
the few products and sums around it every fp32 intermediate is within 64 u of
the magnitudes that enter it (128 u where two inverse RMS values enter).  A
column sum of T terms adds at most (T + 16) u of the sum of magnitudes.  bf16
outputs add half a step, 2^-9 of the value's binade, at most 2^-8 of the value.
"""
import pytest
import torch

from gpu_util import requires_gpu

pytestmark = [pytest.mark.gpu, requires_gpu]

U = 2.0 ** -24
STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
EPS = 1e-5


def _inputs(T, H, xt, yt, post, gate, seed, y=True):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rn(*shape, dt=torch.float32, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dt)
    return dict(
        x=rn(T, H, dt=xt, scale=2.0), y=rn(T, H, dt=yt) if y else None,
        post_w=1 + 0.2 * rn(H) if post else None,
        gate={"none": None, "token": rn(T), "channel": rn(H)}[gate], pre_w=1 + 0.2 * rn(H),
        alpha=0.7, do=rn(T, H, dt=torch.bfloat16), ds=rn(T, H, dt=xt))


def _kind(c, gate):
    return {"none": c.COLI_GATE_NONE, "token": c.COLI_GATE_TOKEN,
            "channel": c.COLI_GATE_CHANNEL}[gate]


def _gate(v, gate):
    if gate == "none":
        return 1.0
    g = v["gate"].double()
    return g[:, None] if gate == "token" else g[None, :]


def _reference(v, gate):
    x = v["x"].double()
    mag = x.abs()
    s = x
    if v["y"] is not None:
        n = v["y"].double()
        if v["post_w"] is not None:
            n = n / torch.sqrt((n * n).mean(1, keepdim=True) + EPS) * v["post_w"].double()
        branch = v["alpha"] * _gate(v, gate) * n
        s = x + branch
        mag = mag + branch.abs()
    r = 1 / torch.sqrt((s * s).mean(1, keepdim=True) + EPS)
    return s, s * r * v["pre_w"].double(), mag, r


CASES = [  # T, H, x type, y type, norm after the block, gate
    (1, 6144, torch.bfloat16, torch.float32, True, "token"),
    (5, 256, torch.float32, torch.float32, True, "channel"),
    (37, 1001, torch.bfloat16, torch.bfloat16, True, "token"),
    (300, 8, torch.float32, torch.bfloat16, False, "none"),
    (3, 1, torch.float32, torch.float32, True, "channel"),
    (150, 4104, torch.bfloat16, torch.bfloat16, False, "channel"),
    (2, 16384, torch.bfloat16, torch.bfloat16, True, "channel"),
    (2, 16383, torch.float32, torch.bfloat16, True, "token"),
    (301, 640, torch.bfloat16, torch.float32, True, "none"),
    # many rows: the ring kernels, one and two vectors per thread
    (450, 6144, torch.bfloat16, torch.bfloat16, True, "channel"),
    (1400, 256, torch.float32, torch.bfloat16, False, "token"),
    (461, 4104, torch.float32, torch.float32, True, "none"),
    (700, 8192, torch.bfloat16, torch.bfloat16, True, "token"),
    (1500, 40, torch.bfloat16, torch.float32, True, "channel"),
    (3001, 2048, torch.bfloat16, torch.bfloat16, False, "none"),
    (300, 6144, torch.float32, torch.float32, True, "token"),    # two rows in the ring
    (310, 4096, torch.bfloat16, torch.float32, True, "channel"),
    # rows of 4-value vectors and of single values, over the widths of each form
    (40, 604, torch.float32, torch.bfloat16, True, "channel"),
    (333, 2004, torch.bfloat16, torch.float32, False, "token"),
    (160, 6140, torch.bfloat16, torch.bfloat16, True, "channel"),
    (2, 16380, torch.float32, torch.float32, True, "none"),
    (900, 505, torch.bfloat16, torch.bfloat16, True, "token"),
    (470, 3001, torch.float32, torch.float32, True, "none"),
]


@pytest.mark.parametrize("T,H,xt,yt,post,gate", CASES)
def test_forward(T, H, xt, yt, post, gate):
    from int4_routed_expert_coli_b200 import coli_moe as c
    v = _inputs(T, H, xt, yt, post, gate, seed=T * 7 + H)
    s, o, mag, r = _reference(v, gate)
    for ot in (torch.float32, torch.bfloat16):
        s_out = torch.full((T, H), float("nan"), dtype=xt, device="cuda")
        out = torch.full((T, H), float("nan"), dtype=ot, device="cuda")
        c.coli_moe_block_norm(T, H, v["x"], v["y"], v["post_w"], v["gate"], _kind(c, gate),
                              v["alpha"], v["pre_w"], EPS, s_out, out)
        assert torch.all((s_out.double() - s).abs() <= STEP[xt] * s.abs() + 64 * U * mag)
        tol = STEP[ot] * o.abs() + 128 * U * (mag * r * v["pre_w"].double().abs() + o.abs())
        # the relative error of s's mean of squares
        tol = tol + o.abs() * 128 * U * (mag * mag).mean(1, keepdim=True) * r * r
        assert torch.all((out.double() - o).abs() <= tol)


@pytest.mark.parametrize("T,H", [(9, 520), (1400, 520)])
def test_forward_without_a_block_and_in_place(T, H):
    from int4_routed_expert_coli_b200 import coli_moe as c
    v = _inputs(T, H, torch.float32, torch.float32, False, "none", seed=3, y=False)
    s, o, mag, r = _reference(v, "none")
    out = torch.empty(T, H, device="cuda")
    c.coli_moe_block_norm(T, H, v["x"], None, None, None, c.COLI_GATE_NONE, 1.0, v["pre_w"], EPS,
                          None, out)
    assert torch.all((out.double() - o).abs() <= 256 * U * o.abs())
    # s over x, o over y
    v = _inputs(T, H, torch.float32, torch.float32, True, "token", seed=4)
    s, o, mag, r = _reference(v, "token")
    c.coli_moe_block_norm(T, H, v["x"], v["y"], v["post_w"], v["gate"], c.COLI_GATE_TOKEN,
                          v["alpha"], v["pre_w"], EPS, v["x"], v["y"])
    assert torch.all((v["x"].double() - s).abs() <= 65 * U * mag)
    assert torch.all((v["y"].double() - o).abs() <=
                     256 * U * (mag * r * v["pre_w"].double().abs() + o.abs()))


def test_rows_of_zeros_infinities_and_nan():
    """A zero row stays zero (eps keeps the root finite); an infinity or a NaN
    stays in its own row."""
    from int4_routed_expert_coli_b200 import coli_moe as c
    T, H = 4, 264
    x = torch.ones(T, H, device="cuda")
    x[0] = 0
    x[1, 5] = float("inf")
    x[2, 7] = float("nan")
    o = torch.empty(T, H, device="cuda")
    w = torch.ones(H, device="cuda")
    c.coli_moe_block_norm(T, H, x, None, None, None, c.COLI_GATE_NONE, 1.0, w, EPS, None, o)
    assert torch.all(o[0] == 0)
    assert torch.isnan(o[1, 5]) and torch.all(o[1, :5] == 0)
    assert torch.all(torch.isnan(o[2]))
    assert torch.all((o[3] - 1 / (1 + EPS) ** 0.5).abs() <= 64 * U)


def _backward(c, v, T, H, gate, with_do=True, with_ds=True):
    got = {"dx": torch.full_like(v["x"], float("nan")),
           "dpre_w": torch.full((H,), float("nan"), device="cuda") if with_do else None,
           "dy": None, "dpost_w": None, "dgate": None}
    if v["y"] is not None:
        got["dy"] = torch.full_like(v["y"], float("nan"))
    if v["post_w"] is not None:
        got["dpost_w"] = torch.full((H,), float("nan"), device="cuda")
    if v["gate"] is not None:
        got["dgate"] = torch.full_like(v["gate"], float("nan"))
    ws = torch.empty(c.coli_moe_block_norm_workspace_size(T, H), dtype=torch.uint8, device="cuda")
    c.coli_moe_block_norm_backward(
        T, H, v["do"] if with_do else None, v["ds"] if with_ds else None, v["x"], v["y"],
        v["post_w"], v["gate"], _kind(c, gate), v["alpha"], v["pre_w"], EPS, got["dx"], got["dy"],
        got["dpre_w"], got["dpost_w"], got["dgate"], ws)
    return got


def _reference_backward(v, gate, with_do=True, with_ds=True):
    """Gradients in 64 bits (v['x'] is the stored s) and, for each, the sum of
    the magnitudes of what is added up in it."""
    s = v["x"].double()
    T, H = s.shape
    r = 1 / torch.sqrt((s * s).mean(1, keepdim=True) + EPS)
    ref, mag = {}, {}
    d = torch.zeros_like(s)
    dm = torch.zeros_like(s)
    if with_ds:
        d = d + v["ds"].double()
        dm = dm + v["ds"].double().abs()
    if with_do:
        do = v["do"].double()
        a = do * v["pre_w"].double()
        d = d + r * (a - s * r ** 2 * (a * s).mean(1, keepdim=True))
        dm = dm + r * (a.abs() + s.abs() * r ** 2 * (a * s).abs().mean(1, keepdim=True))
        ref["dpre_w"] = (do * s * r).sum(0)
        mag["dpre_w"] = (do * s * r).abs().sum(0)
    ref["dx"], mag["dx"] = d, dm
    if v["y"] is None:
        return ref, mag
    y, al = v["y"].double(), v["alpha"]
    ry = torch.ones_like(r)
    pw = torch.ones(H, dtype=torch.float64, device="cuda")
    if v["post_w"] is not None:
        ry = 1 / torch.sqrt((y * y).mean(1, keepdim=True) + EPS)
        pw = v["post_w"].double()
    n = y * ry * pw
    if v["gate"] is not None:
        dim = 1 if gate == "token" else 0
        ref["dgate"], mag["dgate"] = al * (d * n).sum(dim), al * (dm * n.abs()).sum(dim)
    g = _gate(v, gate)
    dn = al * g * d
    dnm = al * (g.abs() if gate != "none" else 1.0) * dm
    if v["post_w"] is not None:
        ref["dpost_w"], mag["dpost_w"] = (dn * y * ry).sum(0), (dnm * y.abs() * ry).sum(0)
        b, bm = dn * pw, dnm * pw.abs()
        dn = ry * (b - y * ry ** 2 * (b * y).mean(1, keepdim=True))
        dnm = ry * (bm + y.abs() * ry ** 2 * (bm * y.abs()).mean(1, keepdim=True))
    ref["dy"], mag["dy"] = dn, dnm
    return ref, mag


@pytest.mark.parametrize("T,H,xt,yt,post,gate", CASES)
def test_backward(T, H, xt, yt, post, gate):
    from int4_routed_expert_coli_b200 import coli_moe as c
    v = _inputs(T, H, xt, yt, post, gate, seed=T * 11 + H)
    got = _backward(c, v, T, H, gate)
    ref, mag = _reference_backward(v, gate)
    for k in ref:
        n = T if k in ("dpre_w", "dpost_w") or (k == "dgate" and gate == "channel") else H
        tol = STEP[got[k].dtype] * ref[k].abs() + (256 + (n + 16 if n == T else 74)) * U * mag[k]
        bad = (got[k].double() - ref[k]).abs() - tol
        assert torch.all(bad <= 0), (k, float(bad.max()))
    # the same bits every time
    again = _backward(c, v, T, H, gate)
    for k in ref:
        assert torch.equal(got[k], again[k]), k


@pytest.mark.parametrize("T,H", [(33, 1032), (1500, 264)])
@pytest.mark.parametrize("with_do,with_ds,y", [(True, False, True), (False, True, True),
                                               (True, False, False), (False, True, False)])
def test_backward_of_parts(with_do, with_ds, y, T, H):
    from int4_routed_expert_coli_b200 import coli_moe as c
    v = _inputs(T, H, torch.float32, torch.float32, y, "channel" if y else "none", seed=5, y=y)
    gate = "channel" if y else "none"
    got = _backward(c, v, T, H, gate, with_do, with_ds)
    ref, mag = _reference_backward(v, gate, with_do, with_ds)
    for k in ref:
        tol = U * ref[k].abs() + (400 + T) * U * mag[k]
        assert torch.all((got[k].double() - ref[k]).abs() <= tol), k


@pytest.mark.parametrize("T,H", [(310, 776), (1400, 520)])
def test_backward_over_its_inputs(T, H):
    """dx over d_s and dy over y."""
    from int4_routed_expert_coli_b200 import coli_moe as c
    v = _inputs(T, H, torch.bfloat16, torch.bfloat16, True, "token", seed=6)
    want = _backward(c, v, T, H, "token")
    ws = torch.empty(c.coli_moe_block_norm_workspace_size(T, H), dtype=torch.uint8, device="cuda")
    dpre, dpost, dg = (torch.empty_like(want[k]) for k in ("dpre_w", "dpost_w", "dgate"))
    c.coli_moe_block_norm_backward(T, H, v["do"], v["ds"], v["x"], v["y"], v["post_w"], v["gate"],
                                   c.COLI_GATE_TOKEN, v["alpha"], v["pre_w"], EPS, v["ds"], v["y"],
                                   dpre, dpost, dg, ws)
    assert torch.equal(v["ds"], want["dx"]) and torch.equal(v["y"], want["dy"])
    assert torch.equal(dpre, want["dpre_w"]) and torch.equal(dpost, want["dpost_w"])
    assert torch.equal(dg, want["dgate"])


def test_gradients_against_differences():
    """Central differences of the library's own fp32 forward: a loss of fixed
    random weights on s and o, stepped along a random direction in every input.
    Step h = 2^-6: the loss sums 2 T H terms of magnitude about 1, each within
    200 u, so the quotient carries sqrt(2 T H) 200 u / h ~ 0.04 of rounding at
    T H = 3 * 40; the third-derivative term h^2 / 6 times O(|direction|^3) adds
    a few percent of the derivative's own terms: 2 % of the sum of the
    magnitudes of the derivative's terms covers both."""
    from int4_routed_expert_coli_b200 import coli_moe as c
    T, H = 3, 40
    v = _inputs(T, H, torch.float32, torch.float32, True, "channel", seed=8)
    g = torch.Generator(device="cuda").manual_seed(9)
    ls, lo = (torch.randn(T, H, generator=g, device="cuda") for _ in range(2))
    names = ["x", "y", "post_w", "gate", "pre_w"]
    step = {k: torch.randn(v[k].shape, generator=g, device="cuda") for k in names}

    def loss(h):
        w = {k: v[k] + h * step[k] for k in names}
        s, o = torch.empty(T, H, device="cuda"), torch.empty(T, H, device="cuda")
        c.coli_moe_block_norm(T, H, w["x"], w["y"], w["post_w"], w["gate"], c.COLI_GATE_CHANNEL,
                              v["alpha"], w["pre_w"], EPS, s, o)
        return float((s.double() * ls).sum() + (o.double() * lo).sum()), s

    h = 2.0 ** -6
    slope = (loss(h)[0] - loss(-h)[0]) / (2 * h)
    _, s = loss(0.0)
    got = {k: torch.empty_like(v[k]) for k in names}
    ws = torch.empty(c.coli_moe_block_norm_workspace_size(T, H), dtype=torch.uint8, device="cuda")
    c.coli_moe_block_norm_backward(T, H, lo, ls, s, v["y"], v["post_w"], v["gate"],
                                   c.COLI_GATE_CHANNEL, v["alpha"], v["pre_w"], EPS, got["x"],
                                   got["y"], got["pre_w"], got["post_w"], got["gate"], ws)
    terms = [(got[k].double() * step[k]) for k in names]
    want = float(sum(t.sum() for t in terms))
    size = float(sum(t.abs().sum() for t in terms))
    assert abs(slope - want) <= 0.02 * size, (slope, want, size)


def test_no_tokens():
    from int4_routed_expert_coli_b200 import coli_moe as c
    H = 64
    e = torch.empty(0, H, device="cuda")
    w = torch.ones(H, device="cuda")
    c.coli_moe_block_norm(0, H, e, e, w, None, c.COLI_GATE_NONE, 1.0, w, EPS, e, e)
    a, b, d = (torch.full((H,), 7.0, device="cuda") for _ in range(3))
    c.coli_moe_block_norm_backward(0, H, e, e, e, e, w, w, c.COLI_GATE_CHANNEL, 1.0, w, EPS, e, e,
                                   a, b, d)
    assert torch.all(a == 0) and torch.all(b == 0) and torch.all(d == 0)


def test_on_another_stream_and_replayed():
    """Captured into a graph with its backward, replayed on new inputs."""
    from int4_routed_expert_coli_b200 import coli_moe as c
    T, H = 40, 512
    v = _inputs(T, H, torch.bfloat16, torch.bfloat16, True, "channel", seed=10)
    o = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    s_out = torch.empty_like(v["x"])
    got = {k: torch.empty_like(v[k]) for k in ("x", "y", "post_w", "gate", "pre_w")}
    ws = torch.empty(c.coli_moe_block_norm_workspace_size(T, H), dtype=torch.uint8, device="cuda")

    def both(x, s, o, g):
        c.coli_moe_block_norm(T, H, x, v["y"], v["post_w"], v["gate"], c.COLI_GATE_CHANNEL,
                              v["alpha"], v["pre_w"], EPS, s, o)
        c.coli_moe_block_norm_backward(T, H, o, x, s, v["y"], v["post_w"], v["gate"],
                                       c.COLI_GATE_CHANNEL, v["alpha"], v["pre_w"], EPS, g["x"],
                                       g["y"], g["pre_w"], g["post_w"], g["gate"], ws)

    both(v["x"], s_out, o, got)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(v["x"], s_out, o, got)
    v["x"].copy_(torch.randn(T, H, device="cuda"))
    graph.replay()
    torch.cuda.synchronize()
    want_s, want_o = torch.empty_like(s_out), torch.empty_like(o)
    want = {k: torch.empty_like(t) for k, t in got.items()}
    both(v["x"], want_s, want_o, want)
    assert torch.equal(s_out, want_s) and torch.equal(o, want_o)
    for k in got:
        assert torch.equal(got[k], want[k]), k


def test_one_workspace_from_wide_to_narrow_rows():
    """Sized once, for the widest call; narrow rows have more partial rows."""
    from int4_routed_expert_coli_b200 import coli_moe as c
    T = 1100
    ws = torch.full((c.coli_moe_block_norm_workspace_size(T, 600),), 255, dtype=torch.uint8,
                    device="cuda")                      # (NaN as floats)
    for H in (600, 513, 512, 505, 256, 36):
        v = _inputs(T, H, torch.float32, torch.float32, True, "channel", seed=H)
        ref, mag = _reference_backward(v, "channel")
        got = {k: torch.empty(H, device="cuda") for k in ("dpre_w", "dpost_w", "dgate")}
        c.coli_moe_block_norm_backward(
            T, H, v["do"], v["ds"], v["x"], v["y"], v["post_w"], v["gate"], c.COLI_GATE_CHANNEL,
            v["alpha"], v["pre_w"], EPS, None, None, got["dpre_w"], got["dpost_w"], got["dgate"], ws)
        for k in got:
            tol = U * ref[k].abs() + (256 + T + 16) * U * mag[k]
            assert torch.all((got[k].double() - ref[k]).abs() <= tol), (H, k)


@pytest.mark.parametrize("T,H,dt", [(700, 2048, torch.bfloat16), (600, 6144, torch.float32),
                                    (40, 2048, torch.bfloat16), (300, 3001, torch.float32)])
def test_in_place_gives_the_same_bits(T, H, dt):
    """s over x and o over y; backward, dx over d_s and dy over d_o (all of one
    type), in the kernels of many and of few rows."""
    from int4_routed_expert_coli_b200 import coli_moe as c
    v = _inputs(T, H, dt, dt, True, "channel", seed=T + H)
    v["do"] = v["do"].to(dt)
    s, o = torch.empty_like(v["x"]), torch.empty_like(v["y"])
    args = (v["post_w"], v["gate"], c.COLI_GATE_CHANNEL, v["alpha"], v["pre_w"], EPS)
    c.coli_moe_block_norm(T, H, v["x"], v["y"], *args, s, o)
    x, y = v["x"].clone(), v["y"].clone()
    c.coli_moe_block_norm(T, H, x, y, *args, x, y)
    assert torch.equal(x, s) and torch.equal(y, o)
    want = _backward(c, v, T, H, "channel")
    ws = torch.empty(c.coli_moe_block_norm_workspace_size(T, H), dtype=torch.uint8, device="cuda")
    col = [torch.empty_like(want[k]) for k in ("dpre_w", "dpost_w", "dgate")]
    do, ds = v["do"].clone(), v["ds"].clone()
    c.coli_moe_block_norm_backward(T, H, do, ds, v["x"], v["y"], *args, ds, do, *col, ws)
    assert torch.equal(ds, want["dx"]) and torch.equal(do, want["dy"])
    for t, k in zip(col, ("dpre_w", "dpost_w", "dgate")):
        assert torch.equal(t, want[k]), k
