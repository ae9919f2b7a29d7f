"""Cases that measure three operators of the library against plain torch forms.

* the norms around a block with its gate and residual scale, forward
  (``norm``) and backward (``norm_bwd``);
* matrix products of rows grouped by expert, ragged group sizes: forward
  (``mm``), gradient of the rows (``mm_dx``) and of the weights (``mm_dw``);
* the grouped product in 8-bit floating point (e4m3) with one scale per block
  of 128, with the quantisation of its rows (``fp8``).

With ``own`` false, ``run`` computes an operator with elementary torch
operations in 32 bits, rounded once at the end; with ``own`` true it calls the
library.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-5
BLOCK = 128
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -126
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}

# H 6144, I 2048 and 256 experts top-8 are the sizes of the repository's
# benchmark layer; 32 experts are the share of one of eight ranks, 4096 wide
# the stacked gate and up rows of one expert.
LISTED = [
    # one token between two blocks of a decode step: latency
    {"name": "norm_decode", "op": "norm", "T": 1, "H": 6144, "x": "bf16", "y": "f32", "post": True,
     "gate": "token"},
    # the same between two blocks of a prefill
    {"name": "norm_prefill", "op": "norm", "T": 4096, "H": 6144, "x": "bf16", "y": "bf16",
     "post": True, "gate": "channel"},
    # its gradient in a training step
    {"name": "norm_bwd_train", "op": "norm_bwd", "T": 4096, "H": 6144, "x": "bf16", "y": "bf16",
     "post": True, "gate": "channel"},
    # an odd width, fp32 stream, no norm after the block
    {"name": "norm_bwd_odd", "op": "norm_bwd", "T": 333, "H": 1001, "x": "f32", "y": "f32",
     "post": False, "gate": "token"},
    # one token's eight experts: the weights' stream
    {"name": "mm_decode", "op": "mm", "R": 8, "E": 32, "N": 4096, "K": 6144, "skew": 0.0,
     "out": "f32"},
    # a small ragged product
    {"name": "mm_ragged", "op": "mm", "R": 777, "E": 16, "N": 136, "K": 264, "skew": 1.0,
     "out": "f32"},
    # gate and up of a rank's share of a 4096-token prefill
    {"name": "mm_prefill", "op": "mm", "R": 4096, "E": 32, "N": 4096, "K": 6144, "skew": 0.3,
     "out": "bf16"},
    # gradient of the rows and of the weights in a training step
    {"name": "mm_dx_train", "op": "mm_dx", "R": 8192, "E": 32, "N": 4096, "K": 6144, "skew": 0.3,
     "out": "bf16"},
    {"name": "mm_dw_train", "op": "mm_dw", "R": 16384, "E": 32, "N": 4096, "K": 6144, "skew": 0.3,
     "out": "f32"},
    # the 8-bit forms: one token, a prefill's share, a dense layer (the shared
    # expert's down projection over 8192 tokens)
    {"name": "fp8_decode", "op": "fp8", "R": 8, "E": 32, "N": 4096, "K": 6144, "skew": 0.0,
     "out": "f32"},
    {"name": "fp8_prefill", "op": "fp8", "R": 4096, "E": 32, "N": 4096, "K": 6144, "skew": 0.3,
     "out": "bf16"},
    {"name": "fp8_dense", "op": "fp8", "R": 8192, "E": 1, "N": 6144, "K": 2048, "skew": 0.0,
     "out": "bf16"},
]


def listed():
    return [dict(c) for c in LISTED]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the listed ranges: rows 1 to 16384, widths 64 to 6144
    (norm: any width from 33 on, odd ones too), 1 to 64 experts."""
    op = rng.choice(["norm", "norm_bwd", "mm", "mm_dx", "mm_dw", "fp8"])
    if op in ("norm", "norm_bwd"):
        x = rng.choice(["f32", "bf16"])
        return {"op": op, "T": _log_int(rng, 1, 4096),
                "H": min(6144, max(33, _log_int(rng, 4, 768) * 8 + rng.choice([0, 0, 1, 4]))),
                "x": x, "y": rng.choice(["f32", x]), "post": rng.random() < 0.5,
                "gate": rng.choice(["none", "token", "channel"])}
    grain = 16 if op == "fp8" else 8
    N = _log_int(rng, 8, 4096 // 8) * 8
    K = _log_int(rng, 64 // grain, 6144 // grain) * grain
    E = _log_int(rng, 1, 64)
    while E * N * K > 32 * 4096 * 6144:
        E = max(1, E // 2)
    R = _log_int(rng, 1, 16384 if op == "mm_dw" else 8192)
    return {"op": op, "R": R, "E": E, "N": N, "K": K, "skew": rng.choice([0.0, 0.3, 1.0]),
            "out": rng.choice(["f32", "bf16"])}


# ---- inputs -------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) % (2 ** 62))
    return g


def _randn(shape, g, dtype, scale=1.0):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, scale, generator=g)


def _groups(case, seed):
    """Group sizes: a few rows go to experts without replacement (one token's
    top-k), many are drawn from a Zipf-like popularity of exponent `skew`."""
    rng = np.random.RandomState(int(seed) % (2 ** 31))
    R, E = case["R"], case["E"]
    if R <= E and case["skew"] == 0.0:
        counts = np.zeros(E, np.int64)
        counts[rng.permutation(E)[:R]] = 1
        return counts
    p = (1.0 + np.arange(E)) ** -case["skew"]
    return rng.multinomial(R, rng.permutation(p / p.sum()))


def _prepare_norm(case, seed):
    g = _generator(seed)
    T, H = case["T"], case["H"]
    xt, yt = DTYPES[case["x"]], DTYPES[case["y"]]
    st = {"case": case, "y": _randn((T, H), g, yt),
          "post_w": 1.0 + _randn((H,), g, torch.float32, 0.1) if case["post"] else None,
          "pre_w": 1.0 + _randn((H,), g, torch.float32, 0.1), "alpha": 0.5, "gate": None}
    if case["gate"] != "none":
        n = T if case["gate"] == "token" else H
        st["gate"] = torch.sigmoid(_randn((n,), g, torch.float32))
    if case["op"] == "norm":
        st["x"] = _randn((T, H), g, xt, 2.0)
    else:
        st["s"] = _randn((T, H), g, xt, 2.0)
        st["do"] = _randn((T, H), g, torch.bfloat16, 1.0)
        st["ds"] = _randn((T, H), g, xt, 1.0)
    if case["op"] == "norm":
        st["s_out"] = torch.empty((T, H), dtype=xt, device="cuda")
        st["o"] = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    st["ws"] = torch.zeros(_WS_HEADER + 4 * 3 * H * 512, dtype=torch.uint8, device="cuda") \
        if case["op"] == "norm_bwd" else None
    return st


_WS_HEADER = 16384


def _prepare_mm(case, seed):
    g = _generator(seed)
    R, E, N, K = case["R"], case["E"], case["N"], case["K"]
    counts = _groups(case, seed)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    active = np.flatnonzero(counts)
    slot = np.repeat(np.arange(len(active)), counts[active])
    inside = np.arange(R) - offsets[:-1][active][slot]
    st = {"case": case,
          "offsets": torch.from_numpy(offsets.astype(np.int32)).cuda(),
          # for the plain form: the active experts, each row's place in a padded
          # [active, longest] array
          "active": torch.from_numpy(active).cuda(), "longest": int(counts.max()),
          "place": torch.from_numpy(slot * int(counts.max()) + inside).cuda(),
          # a user keeps one workspace (cleared once) for the calls of a stream
          "ws": torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")}
    if case["op"] == "fp8":
        st["x"] = _randn((R, K), g, torch.bfloat16)
        wq = torch.empty((E, N, K), dtype=torch.float8_e4m3fn, device="cuda")
        for e in range(E):
            wq[e] = _randn((N, K), g, torch.bfloat16, 100.0).clamp_(-E4M3_MAX, E4M3_MAX)
        st["wq"] = wq
        nb, kb = -(-N // BLOCK), -(-K // BLOCK)
        st["w_scale"] = torch.empty((E, nb, kb), device="cuda").uniform_(1e-4, 4e-4, generator=g)
        st["xq"] = torch.empty((R, K), dtype=torch.float8_e4m3fn, device="cuda")
        st["x_scale"] = torch.empty((kb, R), device="cuda")
    else:
        if case["op"] != "mm_dx":
            st["x"] = _randn((R, K), g, torch.bfloat16)
        if case["op"] != "mm":
            st["dy"] = _randn((R, N), g, torch.bfloat16)
        if case["op"] != "mm_dw":
            st["w"] = _randn((E, N, K), g, torch.bfloat16, 0.02)
    shape = {"mm": (R, N), "fp8": (R, N), "mm_dx": (R, K), "mm_dw": (E, N, K)}[case["op"]]
    st["result"] = torch.empty(shape, dtype=DTYPES[case["out"]], device="cuda")
    return st


def prepare(case, seed):
    return (_prepare_norm if case["op"].startswith("norm") else _prepare_mm)(case, seed)


# ---- the plain forms ------------------------------------------------------------

def _rstd(v):
    return torch.rsqrt(v.square().mean(dim=1, keepdim=True) + EPS)


def _gate(st):
    if st["gate"] is None:
        return 1.0
    return st["gate"][:, None] if st["case"]["gate"] == "token" else st["gate"][None, :]


def _plain_norm(st):
    xt = st["x"].dtype
    x, y = st["x"].float(), st["y"].float()
    n = y * _rstd(y) * st["post_w"] if st["post_w"] is not None else y
    s = x + st["alpha"] * _gate(st) * n
    return {"s": s.to(xt), "o": (s * _rstd(s) * st["pre_w"]).bfloat16()}


def _plain_norm_bwd(st):
    s, y, do = st["s"].float(), st["y"].float(), st["do"].float()
    r = _rstd(s)
    a = do * st["pre_w"]
    d = st["ds"].float() + r * (a - s * r.square() * (a * s).mean(dim=1, keepdim=True))
    got = {"dx": d.to(st["s"].dtype), "dpre_w": (do * s * r).sum(dim=0)}
    ry = _rstd(y) if st["post_w"] is not None else None
    n = y * ry * st["post_w"] if ry is not None else y
    if st["gate"] is not None:
        got["dgate"] = st["alpha"] * (d * n).sum(dim=1 if st["case"]["gate"] == "token" else 0)
    dn = st["alpha"] * _gate(st) * d
    if ry is not None:
        got["dpost_w"] = (dn * y * ry).sum(dim=0)
        b = dn * st["post_w"]
        dn = ry * (b - y * ry.square() * (b * y).mean(dim=1, keepdim=True))
    got["dy"] = dn.to(st["y"].dtype)
    return got


def _padded(st, rows):
    """Rows of the active experts as [active, longest, width], zeros behind each."""
    n = st["active"].numel() * st["longest"]
    out = torch.zeros((n, rows.shape[1]), device=rows.device)
    out[st["place"]] = rows
    return out.view(st["active"].numel(), st["longest"], rows.shape[1])


def _unpadded(st, padded):
    return padded.reshape(-1, padded.shape[2])[st["place"]]


def _plain_mm(st):
    op, out = st["case"]["op"], DTYPES[st["case"]["out"]]
    if op == "mm":
        w = st["w"][st["active"]].float()
        return _unpadded(st, torch.bmm(_padded(st, st["x"].float()), w.mT)).to(out)
    if op == "mm_dx":
        w = st["w"][st["active"]].float()
        return _unpadded(st, torch.bmm(_padded(st, st["dy"].float()), w)).to(out)
    dw = torch.zeros(st["result"].shape, dtype=out, device="cuda")
    dw[st["active"]] = torch.bmm(_padded(st, st["dy"].float()).mT,
                                 _padded(st, st["x"].float())).to(out)
    return dw


def _blocks(t):
    """The last axis padded to whole blocks: [..., blocks, 128]."""
    t = torch.nn.functional.pad(t, (0, -t.shape[-1] % BLOCK))
    return t.view(*t.shape[:-1], -1, BLOCK)


def _plain_fp8(st):
    K, N = st["case"]["K"], st["case"]["N"]
    x = _blocks(st["x"].float())
    top = x.abs().amax(dim=2)
    # a quotient of two tensors: by a plain number, torch multiplies by its
    # rounded reciprocal instead
    scale = (top / torch.full_like(top, E4M3_MAX)).clamp_min(SCALE_MIN)
    q = (x / scale[:, :, None]).to(torch.float8_e4m3fn)
    rows = (q.float() * scale[:, :, None]).view(x.shape[0], -1)[:, :K]
    ws = st["w_scale"][st["active"]].repeat_interleave(BLOCK, dim=1)[:, :N]
    w = (_blocks(st["wq"][st["active"]].float()) * ws[..., None]).flatten(2)[:, :, :K]
    y = _unpadded(st, torch.bmm(_padded(st, rows), w.mT)).to(DTYPES[st["case"]["out"]])
    q = q.view(x.shape[0], -1)[:, :K].contiguous()
    return {"y": y, "q": q, "scale": scale.T.contiguous()}


# ---- one pass ---------------------------------------------------------------------

def _own_run(st):
    from int4_routed_expert_coli_b200 import coli_moe as c
    case = st["case"]
    op = case["op"]
    if op.startswith("norm"):
        T, H = case["T"], case["H"]
        kind = {"none": c.COLI_GATE_NONE, "token": c.COLI_GATE_TOKEN,
                "channel": c.COLI_GATE_CHANNEL}[case["gate"]]
        if op == "norm":
            c.coli_moe_block_norm(T, H, st["x"], st["y"], st["post_w"], st["gate"], kind,
                                  st["alpha"], st["pre_w"], EPS, st["s_out"], st["o"])
            return {"s": st["s_out"], "o": st["o"]}
        got = {"dx": torch.empty_like(st["s"]), "dy": torch.empty_like(st["y"]),
               "dpre_w": torch.empty_like(st["pre_w"])}
        if case["post"]:
            got["dpost_w"] = torch.empty_like(st["post_w"])
        if st["gate"] is not None:
            got["dgate"] = torch.empty_like(st["gate"])
        c.coli_moe_block_norm_backward(T, H, st["do"], st["ds"], st["s"], st["y"], st["post_w"],
                                       st["gate"], kind, st["alpha"], st["pre_w"], EPS, got["dx"],
                                       got["dy"], got["dpre_w"], got.get("dpost_w"),
                                       got.get("dgate"), st["ws"])
        return got
    R, E, N, K = case["R"], case["E"], case["N"], case["K"]
    if op == "mm":
        c.coli_moe_grouped_mm(R, E, N, K, st["x"], st["w"], st["offsets"], st["result"], st["ws"])
    elif op == "mm_dx":
        c.coli_moe_grouped_mm_dx(R, E, N, K, st["dy"], st["w"], st["offsets"], st["result"],
                                 st["ws"])
    elif op == "mm_dw":
        c.coli_moe_grouped_mm_dw(R, E, N, K, st["dy"], st["x"], st["offsets"], st["result"], False,
                                 st["ws"])
    else:
        c.coli_moe_fp8_quantize_rows(R, K, st["x"], st["xq"], st["x_scale"])
        c.coli_moe_fp8_grouped_mm(R, E, N, K, st["xq"], st["x_scale"], st["wq"], st["w_scale"],
                                  st["offsets"], st["result"], st["ws"])
        return {"y": st["result"], "q": st["xq"], "scale": st["x_scale"]}
    return st["result"]


def run(state):
    if own:
        return _own_run(state)
    op = state["case"]["op"]
    if op == "norm":
        return _plain_norm(state)
    if op == "norm_bwd":
        return _plain_norm_bwd(state)
    return _plain_fp8(state) if op == "fp8" else _plain_mm(state)


# ---- cost ---------------------------------------------------------------------------

def _active(case):
    """Experts that get rows: the rows' number bounds it (many rows: all)."""
    return min(case["R"], case["E"])


def work(case):
    size = {"f32": 4, "bf16": 2}
    if case["op"].startswith("norm"):
        T, H, x, y = case["T"], case["H"], size[case["x"]], size[case["y"]]
        gate = {"none": 0, "token": T, "channel": H}[case["gate"]]
        vec = 4 * (H * (2 if case["post"] else 1) + gate)
        if case["op"] == "norm":
            return {"bytes": T * H * (2 * x + y + 2) + vec, "flops": 12 * T * H}
        return {"bytes": T * H * (3 * x + 2 * y + 2) + 2 * vec, "flops": 30 * T * H}
    R, N, K, out = case["R"], case["N"], case["K"], size[case["out"]]
    A = _active(case)
    flops = 2 * R * N * K
    if case["op"] == "fp8":
        kb = -(-K // BLOCK)
        return {"bytes": R * K * 2 + R * K + 4 * kb * R + A * N * K + 4 * A * -(-N // BLOCK) * kb
                + R * N * out, "flops": flops}
    if case["op"] == "mm":
        return {"bytes": 2 * R * K + 2 * A * N * K + R * N * out, "flops": flops}
    if case["op"] == "mm_dx":
        return {"bytes": 2 * R * N + 2 * A * N * K + R * K * out, "flops": flops}
    return {"bytes": 2 * R * (N + K) + case["E"] * N * K * out, "flops": flops}


# ---- the definitions in 64 bits -------------------------------------------------------

def _exact_norm(case, st):
    y = st["y"].double()
    T, H = y.shape
    alpha = st["alpha"]
    g = torch.ones((T, H), dtype=torch.float64, device=y.device)
    if case["gate"] == "token":
        g *= st["gate"].double().unsqueeze(1)
    elif case["gate"] == "channel":
        g *= st["gate"].double()
    hat = y / torch.sqrt((y * y).sum(1) / H + EPS).unsqueeze(1) if case["post"] else y
    wpost = st["post_w"].double() if case["post"] else torch.ones(H, dtype=y.dtype, device=y.device)
    wpre = st["pre_w"].double()
    if case["op"] == "norm":
        s = st["x"].double() + alpha * g * hat * wpost
        return {"s": s, "o": s / torch.sqrt((s * s).sum(1) / H + EPS).unsqueeze(1) * wpre}
    # chain rule through autograd of the definition in 64 bits
    leaves = {"s": st["s"].double(), "y": y, "wpre": wpre, "wpost": wpost, "gate": None}
    if st["gate"] is not None:
        leaves["gate"] = st["gate"].double()
    for t in leaves.values():
        if t is not None:
            t.requires_grad_(True)
    s = leaves["s"]
    o = s / torch.sqrt((s * s).sum(1) / H + EPS).unsqueeze(1) * leaves["wpre"]
    ds, dwpre = torch.autograd.grad(o, [s, leaves["wpre"]], st["do"].double())
    ds = ds + st["ds"].double()
    yl = leaves["y"]
    n = yl
    if case["post"]:
        n = yl / torch.sqrt((yl * yl).sum(1) / H + EPS).unsqueeze(1) * leaves["wpost"]
    branch = alpha * n
    if case["gate"] == "token":
        branch = branch * leaves["gate"].unsqueeze(1)
    elif case["gate"] == "channel":
        branch = branch * leaves["gate"]
    want = {"dy": yl}
    if case["post"]:
        want["dpost_w"] = leaves["wpost"]
    if st["gate"] is not None:
        want["dgate"] = leaves["gate"]
    got = dict(zip(want, torch.autograd.grad(branch, list(want.values()), ds)))
    got["dx"] = ds
    got["dpre_w"] = dwpre
    return got


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"].startswith("norm"):
        return _exact_norm(case, st)
    off = st["offsets"].tolist()
    shape = st["result"].shape
    out = torch.zeros(shape, dtype=torch.float64, device="cuda")
    rows = scale = None
    if case["op"] == "fp8":
        R, K, N = case["R"], case["K"], case["N"]
        kb = -(-K // BLOCK)
        x = st["x"].double()
        rows = torch.empty_like(x)
        scale = torch.empty((kb, R), dtype=torch.float64, device="cuda")
        for b in range(kb):
            part = x[:, b * BLOCK:(b + 1) * BLOCK]
            scale[b] = part.abs().max(dim=1).values / E4M3_MAX
            # by definition the scale and the quotient are fp32 numbers (quotients
            # of bf16 values often fall on the middle of two 8-bit values)
            s = scale[b].clamp(min=SCALE_MIN).float().double().unsqueeze(1)
            q = (part / s).float().to(torch.float8_e4m3fn)
            rows[:, b * BLOCK:(b + 1) * BLOCK] = q.double() * s
        scale.clamp_(min=SCALE_MIN)
    for e in range(case["E"]):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        if case["op"] == "mm":
            out[lo:hi] = st["x"][lo:hi].double() @ st["w"][e].double().T
        elif case["op"] == "mm_dx":
            out[lo:hi] = st["dy"][lo:hi].double() @ st["w"][e].double()
        elif case["op"] == "mm_dw":
            out[e] = st["dy"][lo:hi].double().T @ st["x"][lo:hi].double()
        else:
            w = st["wq"][e].double()
            for n in range(0, N, BLOCK):
                for k in range(0, K, BLOCK):
                    w[n:n + BLOCK, k:k + BLOCK] *= st["w_scale"][e, n // BLOCK, k // BLOCK].double()
            out[lo:hi] = rows[lo:hi] @ w.T
    if case["op"] == "fp8":
        # the 8-bit values themselves are a rounding, not a real number
        return {"y": out, "q": None, "scale": scale}
    return out
