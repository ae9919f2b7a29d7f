"""Refusals of the norm, grouped-product and 8-bit calls: found on the host,
before any CUDA call, so they need no GPU."""
import ctypes

import pytest
import torch

P = ctypes.c_void_p
A = 4096          # a 256-byte aligned address; nothing is read through it


def _lib():
    from int4_routed_expert_coli_b200 import coli_moe as c
    return c, c.lib


def _norm(L, T=4, H=64, x=A, xd=0, y=A, yd=0, post=A, gate=None, kind=0, alpha=1.0, pre=A,
          eps=1e-5, s=A, o=A, od=0):
    return L.coli_moe_block_norm(T, H, P(x), xd, P(y), yd, P(post), P(gate), kind, alpha, P(pre),
                                 eps, P(s), P(o), od, None)


def test_block_norm_refusals():
    c, L = _lib()
    bad, shape, align = c.COLI_ERR_INVALID_ARG, c.COLI_ERR_SHAPE, c.COLI_ERR_ALIGN
    assert _norm(L, T=-1) == bad
    assert _norm(L, H=0) == bad
    assert _norm(L, H=16385) == shape
    assert _norm(L, T=(1 << 24) + 1) == shape
    assert _norm(L, eps=-1.0) == bad
    assert _norm(L, eps=float("nan")) == bad
    assert _norm(L, kind=3) == bad
    assert _norm(L, kind=1) == bad                    # a kind without a gate
    assert _norm(L, gate=A) == bad                    # a gate without a kind
    assert _norm(L, y=None) == bad                    # post_w without a block output
    assert _norm(L, y=None, post=None, gate=A, kind=1) == bad
    assert _norm(L, s=None, o=None) == bad
    assert _norm(L, pre=None) == bad
    assert _norm(L, x=None) == bad
    for k in ("xd", "yd", "od"):
        assert _norm(L, **{k: 2}) == bad
    for k in ("x", "y", "post", "pre", "s", "o"):
        assert _norm(L, **{k: A + 8}) == align
    assert _norm(L, T=0, x=None, y=None, s=None, o=None) == c.COLI_OK


def _bwd(L, T=4, H=64, go=A, od=0, gs=A, s=A, xd=0, y=A, yd=0, post=A, gate=A, kind=1, pre=A,
         eps=1e-5, dx=A, dy=A, dpre=A, dpost=A, dgate=A, ws=A, n=1 << 40):
    return L.coli_moe_block_norm_backward(T, H, P(go), od, P(gs), P(s), xd, P(y), yd, P(post),
                                          P(gate), kind, 1.0, P(pre), eps, P(dx), P(dy), P(dpre),
                                          P(dpost), P(dgate), P(ws), n, None)


def test_block_norm_backward_refusals():
    c, L = _lib()
    bad = c.COLI_ERR_INVALID_ARG
    assert _bwd(L, T=-1) == bad
    assert _bwd(L, H=20000) == c.COLI_ERR_SHAPE
    assert _bwd(L, go=None, gs=None, dpre=None) == bad
    assert _bwd(L, go=None) == bad                    # dpre_w without d_o
    assert _bwd(L, s=None) == bad
    assert _bwd(L, pre=None) == bad
    assert _bwd(L, post=None) == bad                  # dpost_w without post_w
    assert _bwd(L, gate=None, kind=0) == bad          # dgate without a gate
    assert _bwd(L, y=None, post=None, gate=None, kind=0, dpost=None, dgate=None) == bad   # dy
    assert _bwd(L, ws=None) == bad
    assert _bwd(L, ws=A + 16) == c.COLI_ERR_ALIGN
    assert _bwd(L, dx=A + 4) == c.COLI_ERR_ALIGN
    need = L.coli_moe_block_norm_workspace_size(4, 64)
    assert need > 0 and _bwd(L, n=need - 1) == c.COLI_ERR_WORKSPACE
    assert L.coli_moe_block_norm_workspace_size(-1, 64) == 0
    assert L.coli_moe_block_norm_workspace_size(4, 0) == 0


def test_grouped_refusals():
    c, L = _lib()
    big = 1 << 40

    def calls(R=4, E=2, N=64, K=64, a=A, b=A, off=A, out=A, od=0, ws=A, n=big):
        return [f(R, E, N, K, P(a), P(b), P(off), P(out), od, P(ws), n, None)
                for f in (L.coli_moe_grouped_mm, L.coli_moe_grouped_mm_dx)] + \
            [L.coli_moe_grouped_mm_dw(R, E, N, K, P(a), P(b), P(off), P(out), od, 0, P(ws), n, None),
             L.coli_moe_fp8_grouped_mm(R, E, N, K, P(a), P(A), P(b), P(A), P(off), P(out), od, P(ws),
                                       n, None)]

    def all_are(status, **kw):
        assert calls(**kw) == [status] * 4, kw

    bad, shape = c.COLI_ERR_INVALID_ARG, c.COLI_ERR_SHAPE
    all_are(bad, R=-1)
    all_are(bad, E=0)
    all_are(bad, N=0)
    all_are(bad, K=0)
    all_are(shape, E=1025)
    all_are(shape, R=(1 << 24) + 1)
    all_are(shape, N=60)
    all_are(shape, K=60)
    all_are(shape, N=65544)
    all_are(shape, K=65552)
    all_are(bad, od=2)
    for k in ("a", "b", "off", "out", "ws"):
        all_are(bad, **{k: None})
    for k in ("a", "b", "out"):
        all_are(c.COLI_ERR_ALIGN, **{k: A + 8})
    all_are(c.COLI_ERR_ALIGN, off=A + 2)
    all_are(c.COLI_ERR_ALIGN, ws=A + 128)
    all_are(c.COLI_ERR_WORKSPACE, n=L.coli_moe_grouped_workspace_size(4, 2) - 1)
    assert L.coli_moe_grouped_workspace_size(-1, 2) == 0
    assert L.coli_moe_grouped_workspace_size(4, 0) == 0
    # no rows: nothing to do but dw, which needs its output
    st = calls(R=0, a=None, b=None, off=None, out=None, ws=None, n=0)
    assert st == [c.COLI_OK, c.COLI_OK, bad, c.COLI_OK]
    # K of the 8-bit product: multiples of 16
    assert calls(K=72)[3] == shape and calls(K=72, a=None)[0] == bad
    f = L.coli_moe_fp8_grouped_mm
    assert f(4, 2, 64, 64, P(A), None, P(A), P(A), P(A), P(A), 0, P(A), big, None) == bad
    assert f(4, 2, 64, 64, P(A), P(A), P(A), P(A + 4), P(A), P(A), 0, P(A), big,
             None) == c.COLI_ERR_ALIGN


def test_quantize_refusals():
    c, L = _lib()
    f = L.coli_moe_fp8_quantize_rows
    bad = c.COLI_ERR_INVALID_ARG
    assert f(-1, 64, P(A), 0, P(A), P(A), None) == bad
    assert f(4, 0, P(A), 0, P(A), P(A), None) == bad
    assert f(4, 64, P(A), 2, P(A), P(A), None) == bad
    assert f(4, 72, P(A), 0, P(A), P(A), None) == c.COLI_ERR_SHAPE
    assert f(4, 65552, P(A), 0, P(A), P(A), None) == c.COLI_ERR_SHAPE
    assert f(4, 64, None, 0, P(A), P(A), None) == bad
    assert f(4, 64, P(A), 0, None, P(A), None) == bad
    assert f(4, 64, P(A), 0, P(A), None, None) == bad
    assert f(4, 64, P(A + 8), 0, P(A), P(A), None) == c.COLI_ERR_ALIGN
    assert f(0, 64, None, 0, None, None, None) == c.COLI_OK


def test_binding_refuses_host_tensors_and_nothing():
    c, _ = _lib()
    t, w = torch.zeros(2, 64), torch.zeros(64)
    with pytest.raises(ValueError):
        c.coli_moe_block_norm(2, 64, t, None, None, None, c.COLI_GATE_NONE, 1.0, w, 1e-5, t, None)
    with pytest.raises(ValueError):
        c.coli_moe_grouped_mm(2, 1, 64, 64, t.bfloat16(), t.bfloat16(),
                              torch.zeros(2, dtype=torch.int32), t, t)
    with pytest.raises(ValueError):
        c.coli_moe_fp8_quantize_rows(2, 64, t, t, w)
    with pytest.raises(ValueError):
        c.coli_moe_block_norm_backward(0, 64, None, None, None, None, None, None, 0, 1.0, None, 1e-5,
                                       None, None, None, None, None)


def test_binding_refuses_sizes_past_32_bits():
    """They would reach the library as other numbers (2^32 + 2 rows as 2)."""
    c, _ = _lib()
    t, w, big = torch.zeros(2, 64), torch.zeros(64), 2 ** 32 + 2
    with pytest.raises(ValueError, match="32 bits"):
        c.coli_moe_block_norm(big, 64, t, None, None, None, c.COLI_GATE_NONE, 1.0, w, 1e-5, t, None)
    with pytest.raises(ValueError, match="32 bits"):
        c.coli_moe_block_norm_backward(big, 64, t, None, t, None, None, None, c.COLI_GATE_NONE, 1.0,
                                       w, 1e-5, t, None, w, None, None)
    with pytest.raises(ValueError, match="32 bits"):
        c.coli_moe_block_norm_workspace_size(big, 64)
    with pytest.raises(ValueError, match="32 bits"):
        c.coli_moe_grouped_workspace_size(big, 64)
    for f in (c.coli_moe_grouped_mm, c.coli_moe_grouped_mm_dx):
        with pytest.raises(ValueError, match="32 bits"):
            f(big, 1, 64, 64, t, t, w, t, w)
    with pytest.raises(ValueError, match="32 bits"):
        c.coli_moe_grouped_mm_dw(2, 1, big, 64, t, t, w, t, False, w)
    with pytest.raises(ValueError, match="32 bits"):
        c.coli_moe_fp8_quantize_rows(big, 64, t, t, w)
    with pytest.raises(ValueError, match="32 bits"):
        c.coli_moe_fp8_grouped_mm(2, 1, 64, big, t, w, t, w, w, t, w)
    with pytest.raises(TypeError):
        c._ws_arg("workspace", 0)


def test_block_norm_workspace_serves_smaller_calls():
    """The size grows with T and H, so a buffer for (T, H) holds every smaller
    call; and it stays within 1536 rows of H floats behind the header."""
    c, L = _lib()
    size = L.coli_moe_block_norm_workspace_size
    Ts = [1, 2, 148, 443, 444, 445, 739, 740, 741, 768, 769, 887, 888, 889, 1024, 4096, 1 << 24]
    Hs = [1, 33, 64, 256, 505, 511, 512, 513, 520, 600, 852, 853, 854, 888, 1001, 6144, 16384]
    for i, T in enumerate(Ts):
        for j, H in enumerate(Hs):
            n = size(T, H)
            assert n <= c.COLI_WS_HEADER_BYTES + 4 * 1536 * H, (T, H, n)
            if i:
                assert n >= size(Ts[i - 1], H), (T, H)
            if j:
                assert n >= size(T, Hs[j - 1]), (T, H)


def test_grouped_fault_hooks_match_the_header():
    import os
    import re
    c, L = _lib()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = open(os.path.join(root, "include", "coli_moe.h")).read()
    for name in ("COLI_INJECT_WITHHOLD_GROUPED", "COLI_INJECT_SHORT_WAITS"):
        m = re.search(r"#define\s+" + name + r"\s+(\d+)", src)
        assert m and int(m.group(1)) == getattr(c, name)
        assert L.coli_moe_debug_inject(getattr(c, name)) == c.COLI_OK
    assert L.coli_moe_debug_inject(0) == c.COLI_OK
