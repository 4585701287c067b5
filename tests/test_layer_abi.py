"""Host-side checks of the layer operators (no GPU is touched)."""
import ctypes

import numpy as np
import pytest
import torch

from gated_deltanet_chunk_02_b200 import build as B
from gated_deltanet_chunk_02_b200 import gdn
from oracle import layer_oracle as L

FAKE, OUT, ODD = 0x10000, 0x20000, 0x10008     # never dereferenced: every call fails its checks first
BF16, F32 = gdn.GDN_BF16, gdn.GDN_F32


@pytest.fixture(scope="module")
def lib():
    B.build()
    return gdn.load()


def P(x):
    return ctypes.c_void_p(x)


def last(lib):
    return lib.gdn_last_error().decode()


def st(b, h, t):
    return gdn.GdnStrides(b, h, t)


# ---- rotary ----
@pytest.mark.parametrize("rot", [2, 64, 128])
@pytest.mark.parametrize("scaling,factor", [("plain", 1.0), ("linear", 4.0), ("ntk", 8.0),
                                            ("yarn", 8.0)])
def test_frequencies(lib, rot, scaling, factor):
    f, m = gdn.gdn_rotary_frequencies(rot, 10000.0, scaling, factor, 8192)
    g, n = L.rotary_frequencies(rot, 10000.0, scaling, factor, 8192)
    # one rounding to float32 and the powers' own errors in float64
    assert np.allclose(f.numpy(), g, rtol=2.0 ** -23, atol=0)
    assert abs(m - n) <= 2.0 ** -23 * n


@pytest.mark.parametrize("rot,base,scaling,factor,length", [
    (0, 1e4, 0, 1.0, 0), (7, 1e4, 0, 1.0, 0), (130, 1e4, 0, 1.0, 0), (64, 1.0, 0, 1.0, 0),
    (64, float("nan"), 0, 1.0, 0), (64, 1e4, 4, 1.0, 0), (64, 1e4, 1, 0.5, 0),
    (64, 1e4, 3, 2.0, 0)])
def test_frequency_refusals(lib, rot, base, scaling, factor, length):
    out = (ctypes.c_float * 64)()
    m = ctypes.c_float()
    assert lib.gdn_rotary_frequencies(out, ctypes.byref(m), rot, base, scaling, factor,
                                      length) == gdn.GDN_ERR_ARG
    assert lib.gdn_rotary_frequencies(None, ctypes.byref(m), 64, 1e4, 0, 1.0, 0) == gdn.GDN_ERR_ARG


def rotary(lib, q=FAKE, qo=FAKE, qs=None, qos=None, pos=FAKE, inv=FAKE, rot=64, inter=0, back=0,
           B=2, Hq=4, Hk=0, T=8, d=128, dtype=BF16, k=None):
    s = st(4 * 8 * 128, 8 * 128, 128)
    return lib.gdn_rotary(P(q), qs or s, P(qo), qos or s, P(k), s, P(k), s, P(pos), P(inv), 1.0,
                          rot, inter, back, B, Hq, Hk, T, d, dtype, None)


def test_rotary_refusals(lib):
    bad = [dict(rot=0), dict(rot=63), dict(rot=130), dict(inter=2), dict(back=-1), dict(B=-1),
           dict(dtype=7), dict(q=None), dict(qo=None), dict(pos=None), dict(inv=None),
           dict(qs=st(-8, 128, 128)), dict(Hk=1), dict(B=1 << 20, T=1 << 20)]
    for kw in bad:
        assert rotary(lib, **kw) == gdn.GDN_ERR_ARG, kw
    assert rotary(lib, d=64) == gdn.GDN_ERR_UNSUPPORTED
    for kw in [dict(q=ODD), dict(qo=ODD), dict(pos=FAKE + 4), dict(inv=FAKE + 2),
               dict(qs=st(4, 128, 128)), dict(dtype=F32, qs=st(2, 128, 128))]:
        assert rotary(lib, **kw) == gdn.GDN_ERR_ALIGN, kw
    # output rows on one another: broadcast, and a token stride below a row
    assert rotary(lib, qos=st(0, 1024, 128)) == gdn.GDN_ERR_ARG and "overlap" in last(lib)
    assert rotary(lib, qos=st(4096, 1024, 64)) == gdn.GDN_ERR_ARG
    # in place with other strides, and one tensor's output on the other
    assert rotary(lib, qos=st(8192, 1024, 128)) == gdn.GDN_ERR_ARG and "strides" in last(lib)
    for kw in [dict(k=FAKE), dict(k=OUT, qo=OUT)]:
        assert rotary(lib, Hk=4, **kw) == gdn.GDN_ERR_ARG and " is " in last(lib), kw
    # nothing to do
    for kw in [dict(B=0), dict(T=0), dict(Hq=0)]:
        assert rotary(lib, q=None, qo=None, pos=None, inv=None, **kw) == gdn.GDN_OK


# ---- linear attention ----
def shape(B=1, Hk=2, Hv=4, T=100, nseq=0, d=128):
    return gdn.GdnLinearShape(B, Hk, Hv, T, nseq, d)


def forward(lib, q=FAKE, lg=FAKE, s0=None, cu=None, out=OUT, sf=OUT + 64, ws=None, wsb=1 << 40,
            s=None, dtype=BF16):
    return lib.gdn_linear_forward(P(q), P(FAKE), P(FAKE), P(lg), P(s0), P(cu), 1.0, P(out), P(sf),
                                  P(ws), wsb, s or shape(), dtype, None)


def backward(lib, dq=OUT, dk=OUT + 16, cu=None, ws=None, wsb=1 << 40, s=None, ds=None, ds0=None,
             dtype=BF16):
    return lib.gdn_linear_backward(P(FAKE), P(FAKE), P(FAKE), P(FAKE), None, P(FAKE), P(ds), P(cu),
                                   1.0, P(dq), P(dk), P(OUT + 32), P(ds0), P(ws), wsb,
                                   s or shape(), dtype, None)


def test_linear_refusals(lib):
    long = shape(T=65536, Hk=4)
    for f in (forward, backward):
        for kw in [dict(dtype=2), dict(s=shape(B=-1)), dict(s=shape(nseq=-1)),
                   dict(s=shape(Hk=3)), dict(s=shape(Hk=0)), dict(s=shape(Hk=9000, Hv=9000)),
                   dict(s=shape(nseq=2)), dict(s=shape(B=2, nseq=2), cu=FAKE), dict(cu=FAKE),
                   dict(s=shape(B=1 << 20, T=1 << 20)), dict(s=long, wsb=0),
                   dict(s=long, ws=None)]:
            assert f(lib, **kw) == gdn.GDN_ERR_ARG, (f, kw)
        assert f(lib, s=shape(d=64)) == gdn.GDN_ERR_UNSUPPORTED
        assert f(lib, s=shape(nseq=2), cu=FAKE + 2) == gdn.GDN_ERR_ALIGN
        assert f(lib, s=shape(B=0)) == gdn.GDN_OK and f(lib, s=shape(Hk=0, Hv=0)) == gdn.GDN_OK
    for kw in [dict(q=None), dict(lg=None)]:
        assert forward(lib, **kw) == gdn.GDN_ERR_ARG
    for kw in [dict(q=ODD), dict(lg=FAKE + 2), dict(s0=ODD), dict(sf=ODD), dict(s=long, ws=ODD)]:
        assert forward(lib, **kw) == gdn.GDN_ERR_ALIGN, kw
    assert backward(lib, dq=None) == gdn.GDN_ERR_ARG
    # an output that is an input, or another output
    for kw in [dict(out=FAKE), dict(sf=FAKE), dict(s0=OUT + 64), dict(sf=OUT)]:
        assert forward(lib, **kw) == gdn.GDN_ERR_ARG and " is " in last(lib), kw
    for kw in [dict(dq=FAKE), dict(dk=OUT), dict(ds=OUT + 64, ds0=OUT + 64)]:
        assert backward(lib, **kw) == gdn.GDN_ERR_ARG and " is " in last(lib), kw
    assert backward(lib, ds0=ODD) == gdn.GDN_ERR_ALIGN


def test_linear_more_heads_than_a_grid(lib):
    for s, cu in [(shape(B=1 << 26, T=0), None), (shape(nseq=1 << 26, T=1), FAKE)]:
        for f in (forward, backward):
            assert f(lib, s=s, cu=cu) == gdn.GDN_ERR_ARG and "too many" in last(lib)


def test_linear_gradients_without_value_heads_are_refused(lib):
    """dQ and dK [B, Hk, T, d] would be left unwritten."""
    assert backward(lib, s=shape(Hk=2, Hv=0)) == gdn.GDN_ERR_ARG and "value heads" in last(lib)
    assert forward(lib, s=shape(Hk=2, Hv=0)) == gdn.GDN_OK


def test_linear_expiry_hook_arguments(lib):
    f = lib.gdn_debug_arm_linear_expiry
    for block, kernel, ms in [(-1, 0, 5.0), (0, 2, 5.0), (0, 0, 0.0), (0, 1, 2500.0),
                              (0, 1, float("nan"))]:
        assert f(block, kernel, ctypes.c_double(ms)) == gdn.GDN_ERR_ARG


def test_linear_workspace_sizes(lib):
    f, b = lib.gdn_linear_forward_workspace_bytes, lib.gdn_linear_backward_workspace_bytes
    for dtype in (BF16, F32):
        assert f(shape(T=1, Hk=4), dtype) == 0 == b(shape(T=128, Hk=4), dtype)
        assert f(shape(T=65536), dtype) % (4 * 65536) == 0 < f(shape(T=65536), dtype)
        # shared heads: float32 dQ and dK of every value head
        assert b(shape(T=128), dtype) >= 2 * 4 * 128 * 128 * 4
        assert f(shape(Hk=3), dtype) == -1 == b(shape(B=2, nseq=1), dtype)


def test_linear_decode_refusals(lib):
    def call(q=FAKE, lg=FAKE, S=OUT + 64, slots=None, nslots=8, B=2, Hk=2, Hv=4, n=1, d=128,
             dtype=BF16):
        return lib.gdn_linear_decode(P(q), P(FAKE), P(FAKE), P(lg), P(S), P(slots), nslots, 1.0,
                                     P(OUT), B, Hk, Hv, n, d, dtype, None)
    for kw in [dict(q=None), dict(lg=None), dict(S=None), dict(nslots=1), dict(Hk=3), dict(Hk=0),
               dict(n=-1), dict(B=65536), dict(dtype=9), dict(slots=FAKE, nslots=-1), dict(S=OUT),
               dict(S=FAKE)]:
        assert call(**kw) == gdn.GDN_ERR_ARG, kw
    for kw in [dict(q=ODD), dict(S=ODD), dict(slots=FAKE + 2), dict(lg=FAKE + 2)]:
        assert call(**kw) == gdn.GDN_ERR_ALIGN, kw
    assert call(d=64) == gdn.GDN_ERR_UNSUPPORTED
    assert call(q=None, B=0) == gdn.GDN_OK == call(q=None, n=0)


# ---- block norm ----
def norm(lib, y=FAKE, ys=None, z=None, wo=FAKE, r=None, wi=None, eps=1e-6, act=1, X=FAKE, N=None,
         B=2, T=4, H=3, d=128, dtype=BF16):
    return lib.gdn_block_norm(P(y), ys or st(4096, 512, 128), P(z), P(wo), P(r), P(wi), 1.0, eps,
                              act, P(X), P(N), B, T, H, d, dtype, None)


def norm_back(lib, z=None, dz=None, wo=FAKE, dwo=FAKE, wi=None, dwi=None, dX=FAKE, dN=None, r=None,
              dr=None, dy=FAKE, dys=None, ws=FAKE, wsb=1 << 40, B=2, T=4, H=3, d=128):
    s = st(4096, 512, 128)
    return lib.gdn_block_norm_backward(P(FAKE), s, P(z), P(wo), P(r), P(wi), P(dX), P(dN), 1.0,
                                       1e-6, 0, P(dy), dys or s, P(dz), P(dr), P(dwo), P(dwi),
                                       P(ws), wsb, B, T, H, d, BF16, None)


def test_norm_refusals(lib):
    for kw in [dict(y=None), dict(eps=0.0), dict(eps=float("nan")), dict(act=2), dict(X=None),
               dict(wi=FAKE), dict(N=FAKE), dict(dtype=3), dict(T=-1), dict(ys=st(-8, 8, 8))]:
        assert norm(lib, **kw) == gdn.GDN_ERR_ARG, kw
    for kw in [dict(d=64), dict(H=1, d=12), dict(H=129), dict(H=1, d=16392)]:
        assert norm(lib, **kw) == gdn.GDN_ERR_UNSUPPORTED, kw
    for kw in [dict(y=ODD), dict(z=ODD), dict(wo=ODD), dict(r=ODD), dict(X=ODD),
               dict(ys=st(4096, 512, 4))]:
        assert norm(lib, **kw) == gdn.GDN_ERR_ALIGN, kw
    # an output that is an input (but for X and R), or the other output
    for kw in [dict(), dict(X=OUT, z=OUT), dict(X=OUT, N=OUT, wi=FAKE),
               dict(X=OUT, N=OUT + 64, wi=FAKE, r=OUT + 64)]:
        assert norm(lib, **kw) == gdn.GDN_ERR_ARG and " is " in last(lib), kw
    for kw in [dict(B=0), dict(T=0), dict(H=0)]:
        assert norm(lib, y=None, **kw) == gdn.GDN_OK


def test_norm_backward_refusals(lib):
    for kw in [dict(z=FAKE), dict(dz=FAKE), dict(dwo=None), dict(wi=FAKE), dict(dN=FAKE),
               dict(dr=FAKE), dict(dX=None), dict(dy=None), dict(wsb=0), dict(ws=None),
               dict(dys=st(0, 512, 128))]:
        assert norm_back(lib, **kw) == gdn.GDN_ERR_ARG, kw
    for kw in [dict(dy=ODD), dict(dwo=ODD), dict(ws=ODD), dict(dX=ODD), dict(dys=st(4096, 512, 4))]:
        assert norm_back(lib, **kw) == gdn.GDN_ERR_ALIGN, kw
    for kw in [dict(), dict(dy=OUT), dict(dy=OUT, dwo=OUT), dict(dy=OUT, dwo=OUT + 64, dX=OUT),
               dict(dy=OUT, dwo=OUT + 64, r=OUT + 128, dr=OUT + 128)]:
        assert norm_back(lib, **kw) == gdn.GDN_ERR_ARG and " is " in last(lib), kw
    assert norm_back(lib, wo=None, dwo=None, B=0) == gdn.GDN_OK
    f = lib.gdn_block_norm_backward_workspace_bytes
    assert f(2, 4, 3, 128) > 0 and f(0, 4, 3, 128) == 0 and f(1, 1, 1, 12) == -1


# ---- outputs on a part of an input, or of one another ----
FAR = [0x1000000 * i for i in range(1, 24)]    # 16 MiB apart; never dereferenced


def shares(lib, rc):
    return rc == gdn.GDN_ERR_ARG and "shares memory" in last(lib)


def test_rotary_outputs_on_parts_of_others(lib):
    """[2, 4, 8, 128] bf16: 128 KiB each; the fused layout [2, 8, 12, 128]."""
    s, f = st(4096 * 2, 1024, 128), st(8 * 12 * 128, 128, 12 * 128)

    def call(q=FAR[0], qs=s, qo=FAR[1], qos=s, k=FAR[2], ks=s, ko=FAR[3], kos=s, pos=FAR[4],
             inv=FAR[5]):
        return lib.gdn_rotary(P(q), qs, P(qo), qos, P(k), ks, P(ko), kos, P(pos), P(inv), 1.0, 64, 0,
                              0, 2, 4, 4, 8, 128, BF16, None)
    end = 2 * 8192 + 0                                 # bytes of the first batch row
    for kw in [dict(qo=FAR[0] + 256), dict(qo=FAR[0] - 256), dict(qo=FAR[2] + end),
               dict(ko=FAR[1] + 16), dict(ko=FAR[0] + 1024), dict(ko=FAR[4]),
               dict(qo=FAR[5] - 16 * 1024),
               # a head further on in the fused layout; K's output on Q's last head in place
               dict(q=FAR[0], qs=f, qo=FAR[0] + 256, qos=f),
               dict(q=FAR[0], qs=f, qo=FAR[0], qos=f, k=FAR[2], ko=FAR[0] + 3 * 256, kos=f)]:
        assert shares(lib, call(**kw)), kw


def test_linear_outputs_on_parts_of_others(lib):
    def fwd(out=FAR[0], sf=FAR[1], s0=FAR[2], lg=FAR[3], q=FAR[4], ws=FAR[12], s=shape(), cu=None):
        return lib.gdn_linear_forward(P(q), P(FAR[5]), P(FAR[6]), P(lg), P(s0), P(cu), 1.0, P(out),
                                      P(sf), P(ws), 1 << 40, s, BF16, None)

    def bwd(dq=FAR[0], dk=FAR[1], dv=FAR[2], ds0=FAR[3], do=FAR[4], ds=FAR[5], ws=FAR[12]):
        return lib.gdn_linear_backward(P(FAR[6]), P(FAR[7]), P(FAR[8]), P(FAR[9]), P(FAR[10]), P(do),
                                       P(ds), None, 1.0, P(dq), P(dk), P(dv), P(ds0), P(ws), 1 << 40,
                                       shape(), BF16, None)

    def dec(out=FAR[0], S=FAR[1], q=FAR[2], slots=FAR[4]):
        return lib.gdn_linear_decode(P(q), P(FAR[5]), P(FAR[6]), P(FAR[7]), P(S), P(slots), 9, 1.0,
                                     P(out), 2, 2, 4, 1, 128, BF16, None)
    long = shape(T=65536, Hk=4)                        # its states take more than a megabyte
    for kw in [dict(out=FAR[4] + 16), dict(out=FAR[6] - 16), dict(sf=FAR[2] + 65536),
               dict(out=FAR[1] - 256), dict(sf=FAR[3] - 16), dict(s=long, ws=FAR[1] - 65536),
               dict(s=shape(nseq=3), cu=FAR[0] + 64)]:
        assert shares(lib, fwd(**kw)), kw
    for kw in [dict(dq=FAR[6] + 16), dict(dk=FAR[0] + 1024), dict(dv=FAR[4] - 16),
               dict(ds0=FAR[5] + 65536), dict(ws=FAR[8] - 65536), dict(ws=FAR[1])]:
        assert shares(lib, bwd(**kw)), kw
    # a pool of 9 x 4 states is 2.25 MiB
    for kw in [dict(S=FAR[0] - (9 << 18) + 16), dict(out=FAR[2] + 16), dict(S=FAR[4] - 65536)]:
        assert shares(lib, dec(**kw)), kw


def test_norm_outputs_on_parts_of_others(lib):
    """[2, 4, 384] bf16 rows: 6 KiB each; Y is [2, 3, 4, 128]."""
    s = st(1536, 512, 128)

    def fwd(y=FAR[0], z=FAR[1], wo=FAR[2], r=FAR[3], wi=FAR[4], X=FAR[5], N=FAR[6]):
        return lib.gdn_block_norm(P(y), s, P(z), P(wo), P(r), P(wi), 1.0, 1e-6, 1, P(X), P(N), 2, 4, 3,
                                  128, BF16, None)

    def bwd(dX=FAR[7], dN=FAR[8], dy=FAR[9], dz=FAR[10], dr=FAR[11], dwo=FAR[12], dwi=FAR[13],
            ws=FAR[14]):
        return lib.gdn_block_norm_backward(P(FAR[0]), s, P(FAR[1]), P(FAR[2]), P(FAR[3]), P(FAR[4]),
                                           P(dX), P(dN), 1.0, 1e-6, 1, P(dy), s, P(dz), P(dr), P(dwo),
                                           P(dwi), P(ws), 1 << 40, 2, 4, 3, 128, BF16, None)
    for kw in [dict(X=FAR[0] + 16), dict(X=FAR[3] + 768), dict(r=FAR[5] + 16), dict(N=FAR[5] + 768),
               dict(N=FAR[1] - 16), dict(X=FAR[2] - 16), dict(N=FAR[4] + 512)]:
        assert shares(lib, fwd(**kw)), kw
    for kw in [dict(dy=FAR[0] + 256), dict(dz=FAR[1] + 16), dict(dr=FAR[7] + 768), dict(dy=FAR[7] - 16),
               dict(dwo=FAR[13] - 512), dict(dr=FAR[9] + 16), dict(ws=FAR[12] - 512),
               dict(dz=FAR[8] + 6128), dict(dwi=FAR[4] + 16)]:
        assert shares(lib, bwd(**kw)), kw


# ---- the binding ----
def test_binding_refuses_what_the_library_cannot_see(lib):
    x = torch.zeros(1, 2, 4, 128, dtype=torch.bfloat16)
    lg = torch.zeros(2)
    S = torch.zeros(1, 2, 128, 128)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.gdn_linear_decode(x, x, x, lg, S, x.clone())
    with pytest.raises(ValueError, match="shares memory"):
        gdn.gdn_linear_decode(x, x, x, lg, S, x)
    with pytest.raises(ValueError, match="shares memory"):
        gdn.gdn_linear_forward(x, x, x, lg, S, x.clone(), S, None)
    with pytest.raises(ValueError, match="cu_seqlens"):
        gdn.gdn_linear_forward(x, x, x, lg, None, x.clone(), None, None,
                               cu_seqlens=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(TypeError):
        gdn.gdn_rotary(x, None, None, torch.ones(4), None, None)
    with pytest.raises(KeyError):
        gdn.gdn_rotary_frequencies(64, scaling="other")
    with pytest.raises(gdn.GdnError):
        gdn.gdn_rotary_frequencies(63)
