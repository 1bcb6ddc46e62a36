"""Refusals of the gated delta rule's and the root-mean-square norm's entry points, without a GPU: every
call here fails validation before anything is enqueued, or has nothing to enqueue."""
import ctypes

import pytest
import torch

from linear_recurrent_token_b200 import mlstm

A = [0x1000000 * (i + 1) for i in range(24)]  # fake, aligned, never dereferenced
P = ctypes.c_void_p
NULL, SHAPE, DTYPE, ALIGN, WORKSPACE, ALIAS = 1, 2, 3, 4, 5, 7


def dense(H, T, D):
    return mlstm.GdrStride(H * T * D, T * D, D)


def gdr(B=1, HK=1, H=2, T=8, K=16, V=16, num_seqs=0, dtype=0, mode=0, **strides):
    s = dict(q=dense(HK, T, K), k=dense(HK, T, K), v=dense(H, T, V), g=mlstm.GdrStride(H * T, T, 1),
             beta=mlstm.GdrStride(H * T, T, 1), o=dense(H, T, V))
    s.update({n: mlstm.GdrStride(*x) for n, x in strides.items()})
    return mlstm.GdrParams(B, HK, H, T, K, V, num_seqs, dtype, mode, s["q"], s["k"], s["v"], s["g"], s["beta"], s["o"])


def fwd(p, S0=None, off=None, S_out=None, ws=None, ws_bytes=0, **kw):
    a = dict(zip(("q", "k", "v", "g", "beta", "o"), A)) | kw
    return mlstm.lib().mlstm_gdr_fwd(ctypes.byref(p), a["q"], a["k"], a["v"], a["g"], a["beta"], S0, off, a["o"], S_out,
                                     ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=65535, T=2**22), SHAPE), (dict(B=-1), SHAPE), (dict(T=-1), SHAPE), (dict(T=2**30 + 1), SHAPE), (dict(K=12), SHAPE), (dict(K=0), SHAPE),
    (dict(K=264), SHAPE), (dict(V=4), SHAPE), (dict(V=0), SHAPE), (dict(HK=3, H=4), SHAPE), (dict(HK=0, H=2), SHAPE),
    (dict(H=65536, HK=1), SHAPE), (dict(B=65536), SHAPE), (dict(dtype=2), DTYPE), (dict(mode=3), SHAPE),
    (dict(K=136, mode=2), SHAPE), (dict(num_seqs=2, B=2), SHAPE), (dict(num_seqs=-1), SHAPE),
    (dict(q=(128, 128, 18)), SHAPE), (dict(v=(256, -128, 16)), SHAPE), (dict(v=(0, 2**51, 16)), SHAPE),
    (dict(g=(0, 0, -1)), SHAPE), (dict(o=(0, 0, 16)), SHAPE), (dict(o=(0, 128, 8)), SHAPE),
])
def test_fwd_refuses_sizes_and_strides(kw, status):
    assert fwd(gdr(**kw)) == status


def test_fwd_refuses_pointers():
    p = gdr(mode=1)
    for n in ("q", "k", "v", "g", "beta", "o"):
        assert fwd(p, **{n: None}) == NULL
    for n in ("q", "k", "v", "o"):
        assert fwd(p, **{n: A[9] + 8}) == ALIGN
    assert fwd(p, g=A[9] + 2) == ALIGN and fwd(p, S0=A[9] + 4) == ALIGN
    assert fwd(p, o=A[0]) == ALIAS and fwd(p, o=A[2] + 64) == ALIAS
    assert fwd(p, S0=A[9], S_out=A[9] + 64) == ALIAS and fwd(p, S_out=A[5]) == ALIAS
    assert fwd(gdr(num_seqs=1)) == NULL  # offsets
    chunk = gdr(mode=2)
    need = mlstm.gdr_fwd_workspace_size(chunk)
    assert need > 0 and mlstm.gdr_fwd_workspace_size(p) == 0
    assert fwd(chunk) == WORKSPACE and fwd(chunk, ws=A[9], ws_bytes=need - 1) == WORKSPACE
    assert fwd(chunk, ws=A[0], ws_bytes=need) == ALIAS
    assert mlstm.lib().mlstm_gdr_fwd(None, *A[:10], 0, None) == NULL


def test_fwd_with_nothing_to_do():
    assert fwd(gdr(B=0)) == 0
    assert fwd(gdr(H=0, HK=0)) == 0
    assert fwd(gdr(T=0), q=None, k=None, v=None, g=None, beta=None, o=None, S0=A[9], S_out=A[9]) == 0
    assert mlstm.gdr_fwd_workspace_size(gdr(T=0, mode=2)) == 0 == mlstm.gdr_bwd_workspace_size(gdr(T=0))


def test_auto_takes_chunks_from_a_length_on():
    size = lambda **kw: mlstm.gdr_fwd_workspace_size(gdr(**kw))
    assert size(T=31) == 0 and size(T=32) > 0 and size(T=4096, K=256) == 0
    # a packed batch may have a ragged chunk for every sequence more
    assert size(T=640, num_seqs=5) > size(T=640)
    assert size(T=640) - size(T=576) == size(T=128) - size(T=64) > 0


def step(B=3, HK=1, H=2, K=16, V=16, pool=3, dtype=0, slots=None, strides=None, **kw):
    s = dict(q=(HK * K, K, 0), k=(HK * K, K, 0), v=(H * V, V, 0), g=(H, 1, 0), beta=(H, 1, 0), o=(H * V, V, 0)) | (strides or {})
    p = mlstm.GdrStepParams(B, HK, H, K, V, pool, dtype, *(mlstm.GdrStride(*s[n]) for n in ("q", "k", "v", "g", "beta", "o")))
    a = dict(zip(("q", "k", "v", "g", "beta", "S", "o"), A)) | kw
    return mlstm.lib().mlstm_gdr_step(ctypes.byref(p), a["q"], a["k"], a["v"], a["g"], a["beta"], slots, a["S"], a["o"], None)


def test_step_refusals():
    assert step(K=260) == SHAPE and step(V=12) == SHAPE and step(dtype=5) == DTYPE and step(pool=-1) == SHAPE
    assert step(pool=2) == SHAPE  # without slots every row needs its state
    assert step(strides=dict(o=(0, 16, 0))) == SHAPE and step(strides=dict(q=(18, 16, 0))) == SHAPE
    for n in ("q", "k", "v", "g", "beta", "S", "o"):
        assert step(**{n: None}) == NULL
    assert step(S=A[9] + 4) == ALIGN and step(slots=A[9] + 2) == ALIGN
    assert step(S=A[0]) == ALIAS and step(o=A[2]) == ALIAS and step(o=A[5]) == ALIAS and step(slots=A[5]) == ALIAS
    assert step(B=0) == 0


def bwd(p, dstrides=None, ws=A[20], ws_bytes=1 << 40, **kw):
    names = ("q", "k", "v", "g", "beta", "S0", "off", "do", "dS", "dq", "dk", "dv", "dg", "dbeta", "dS0")
    a = dict(zip(names, A)) | dict(S0=None, off=None, dS=None, dS0=None) | kw
    s = dstrides or [dense(p.HK, p.T, p.K), dense(p.HK, p.T, p.K), dense(p.H, p.T, p.V)]
    return mlstm.lib().mlstm_gdr_bwd(ctypes.byref(p), *(a[n] for n in names[:9]), *s, *(a[n] for n in names[9:]), ws, ws_bytes, None)


def test_bwd_refusals():
    p = gdr()
    for n in ("q", "k", "v", "g", "beta", "do", "dq", "dk", "dv", "dg", "dbeta"):
        assert bwd(p, **{n: None}) == NULL
    for n in ("q", "dq", "dv", "dS0", "do"):
        assert bwd(p, **{n: A[16] + 8}) == ALIGN
    assert bwd(p, dg=A[16] + 2) == ALIGN
    assert bwd(gdr(K=136)) == SHAPE and bwd(gdr(dtype=9)) == DTYPE
    one = mlstm.GdrStride(0, 0, 16)
    assert bwd(p, dstrides=[dense(1, 8, 16), dense(1, 8, 16), one]) == SHAPE
    assert bwd(p, dq=A[0]) == ALIAS and bwd(p, dk=A[9]) == ALIAS and bwd(p, dS=A[16], dS0=A[16]) == ALIAS
    assert bwd(p, ws_bytes=mlstm.gdr_bwd_workspace_size(p) - 1) == WORKSPACE and bwd(p, ws=None) == WORKSPACE
    assert bwd(p, ws=A[2], ws_bytes=1 << 40) == ALIAS
    assert bwd(gdr(num_seqs=1)) == NULL
    assert bwd(gdr(B=0)) == 0


def rms(rows=4, D=64, dtype=0, quant=0, group=0, eps=1e-6, **kw):
    p = mlstm.RmsParams(rows, D, dtype, quant, group, eps)
    a = dict(x=A[0], residual=None, weight=None, r_out=None, y=A[1], scales=None) | kw
    return mlstm.lib().mlstm_rms_norm(ctypes.byref(p), a["x"], a["residual"], a["weight"], a["r_out"], a["y"], a["scales"], None)


def test_status_refusals():
    L = mlstm.lib()
    many = gdr(B=8, HK=16, H=16, T=64, K=64, V=128, dtype=1, mode=2)
    assert L.mlstm_gdr_status(None, A[0], None) == NULL
    assert L.mlstm_gdr_status(ctypes.byref(gdr(K=12)), A[0], None) == SHAPE
    assert L.mlstm_gdr_status(ctypes.byref(gdr(dtype=3)), A[0], None) == DTYPE
    assert L.mlstm_gdr_status(ctypes.byref(many), None, None) == NULL  # its error word lives there


def test_rms_refusals():
    assert rms(rows=-1) == SHAPE and rms(D=0) == SHAPE and rms(D=16385) == SHAPE and rms(eps=-1.0) == SHAPE
    assert rms(eps=float("nan")) == SHAPE and rms(dtype=2) == DTYPE and rms(quant=3) == DTYPE
    assert rms(quant=1, group=64, scales=A[2]) == SHAPE and rms(rows=2**31) == SHAPE
    assert rms(x=None) == NULL and rms(y=None) == NULL and rms(quant=1) == NULL and rms(residual=A[2]) == NULL
    assert rms(x=A[0] + 4) == ALIGN and rms(weight=A[2] + 8) == ALIGN and rms(quant=1, scales=A[2] + 4) == ALIGN
    assert rms(y=A[0]) == ALIAS and rms(residual=A[2], r_out=A[2] + 64) == ALIAS and rms(residual=A[2], r_out=A[1]) == ALIAS
    assert rms(quant=2, scales=A[1]) == ALIAS
    assert rms(rows=0, x=None, y=None) == 0


def test_rms_bwd_refusals():
    L = mlstm.lib()

    def call(rows=4, D=64, dtype=0, ws=A[5], ws_bytes=1 << 40, **kw):
        p = mlstm.RmsParams(rows, D, dtype, 0, 0, 1e-6)
        a = dict(dy=A[0], r=A[1], weight=None, dres=None, dx=A[2], dw=A[3]) | kw
        return L.mlstm_rms_norm_bwd(ctypes.byref(p), a["dy"], a["r"], a["weight"], a["dres"], a["dx"], a["dw"], ws, ws_bytes, None)

    assert call(D=20000) == SHAPE and call(dtype=3) == DTYPE
    assert call(dy=None) == NULL and call(r=None) == NULL and call(dx=None) == NULL
    assert call(dx=A[1]) == ALIAS and call(dx=A[0] + 16) == ALIAS and call(dw=A[2]) == ALIAS and call(ws=A[1]) == ALIAS
    assert call(dx=A[2] + 8) == ALIGN
    p = mlstm.RmsParams(4, 64, 0, 0, 0, 1e-6)
    need = L.mlstm_rms_norm_bwd_workspace_size(ctypes.byref(p))
    assert need > 0 and call(ws_bytes=need - 1) == WORKSPACE and call(ws=None) == WORKSPACE
    assert call(rows=0, dy=None, r=None, dx=None, dw=None) == 0


def cpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_binding_refuses_before_the_device():
    q, v, g = cpu(2, 1, 5, 16), cpu(2, 2, 5, 8), cpu(2, 2, 5, dtype=torch.float32)
    S = cpu(2, 2, 16, 8, dtype=torch.float32)
    with pytest.raises(ValueError, match="CUDA"):
        mlstm.gdr_fwd(q, q, v, g, g, S)
    with pytest.raises(ValueError, match="k must have shape"):
        mlstm.gdr_fwd(q, cpu(2, 1, 4, 16), v, g, g)
    with pytest.raises(TypeError, match="v must be"):
        mlstm.gdr_fwd(q, q, v.float(), g, g)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        mlstm.gdr_fwd(q.half(), q.half(), v.half(), g, g)
    with pytest.raises(ValueError, match="beta must have shape"):
        mlstm.gdr_fwd(q, q, v, g, g[:, :1])
    with pytest.raises(ValueError, match="S0 must have shape"):
        mlstm.gdr_fwd(q, q, v, g, g, S[:1])
    with pytest.raises(ValueError, match="last axis of q"):
        mlstm.gdr_fwd(cpu(2, 1, 5, 32)[..., ::2], q, v, g, g)
    with pytest.raises(ValueError, match="mode must be"):
        mlstm.gdr_fwd(q, q, v, g, g, mode="fast")
    with pytest.raises(ValueError, match="seq_offsets"):
        mlstm.gdr_fwd(q, q, v, g, g, seq_offsets=torch.zeros(3, dtype=torch.int32))  # two batch rows
    with pytest.raises(TypeError, match="seq_offsets must be"):
        mlstm.gdr_fwd(q[:1], q[:1], v[:1], g[:1], g[:1], seq_offsets=torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="do must have shape"):
        mlstm.gdr_bwd(q, q, v, g, g, v[:1])
    with pytest.raises(ValueError, match="last axis of do"):
        mlstm.gdr_bwd(q, q, v, g, g, cpu(1, 1, 1, 1).expand(2, 2, 5, 8))
    with pytest.raises(ValueError, match="S must have shape"):
        mlstm.gdr_step(q[:, :, 0], q[:, :, 0], v[:, :, 0], g[:, :, 0], g[:, :, 0], S[:, :, :8])
    with pytest.raises(TypeError, match="slots must be"):
        mlstm.gdr_step(q[:, :, 0], q[:, :, 0], v[:, :, 0], g[:, :, 0], g[:, :, 0], S, slots=torch.zeros(2, dtype=torch.int64))
    x = cpu(3, 16)
    with pytest.raises(ValueError, match="contiguous"):
        mlstm.rms_norm(cpu(3, 32)[:, ::2])
    with pytest.raises(ValueError, match="quant must be"):
        mlstm.rms_norm(x, quant="e5m2")
    with pytest.raises(ValueError, match="group must be"):
        mlstm.rms_norm(x, quant="int8", group=16)
    with pytest.raises(ValueError, match="residual_out without"):
        mlstm.rms_norm(x, residual_out=x)
    with pytest.raises(ValueError, match="scales without"):
        mlstm.rms_norm(x, scales=cpu(3, 1, dtype=torch.float32))
    with pytest.raises(TypeError, match="weight must be"):
        mlstm.rms_norm(x, weight=x[0])
    with pytest.raises(ValueError, match="dy must have shape"):
        mlstm.rms_norm_bwd(x[:2], x)
