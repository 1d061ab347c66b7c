"""MXFP4 on the CPU: the oracle's format against its definition, and what the
library and its binding refuse before anything is launched."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from combine_wave_level_amd import moe

FAKE = ctypes.c_void_p(0x10000)   # aligned, never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x10004)


def _p(**kw):
    base = dict(T=4, d=256, I=128, E_global=8, k=2, e_begin=0, E_local=8, experts_per_wave=4,
                x_dtype=moe.MOE_BF16, w_dtype=moe.MOE_BF16, out_dtype=moe.MOE_BF16, activation=moe.MOE_ACT_SWIGLU)
    base.update(kw)
    return moe.Problem(*[base[n] for n, _ in moe.Problem._fields_])


# ------------------------------------------------------------------ the format

def test_e2m1_code_table_and_round_trip():
    vals = oracle.e2m1_decode(np.arange(16, dtype=np.uint8))
    assert vals[:8].tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6] and (vals[8:] == -vals[:8]).all()
    assert oracle.e2m1_encode(vals).tolist() == list(range(16))     # -0 keeps its sign


def test_e2m1_ties_go_to_the_even_code():
    ties = {0.25: 0, 0.75: 2, 1.25: 2, 1.75: 4, 2.5: 4, 3.5: 6, 5.0: 6}
    for v, code in ties.items():
        assert oracle.e2m1_encode(np.array([v, -v])).tolist() == [code, code | 8]
        up, down = np.nextafter(v, 9), np.nextafter(v, 0)
        lo = max(c for c in range(8) if oracle.e2m1_decode(np.uint8(c)) < v)
        assert oracle.e2m1_encode(np.array([up, down])).tolist() == [lo + 1, lo]


def test_block_scale_is_the_smallest_without_saturation():
    rng = np.random.default_rng(3)
    v = rng.standard_normal((50, 64)) * np.exp2(rng.integers(-60, 60, (50, 1)))
    codes, sb, q = oracle.quantize_mxfp4(v)
    s = np.exp2(sb.astype(np.float64) - 127)
    amax = np.abs(v.reshape(50, 2, 32)).max(-1)
    assert (amax <= 6 * s).all() and (amax > 3 * s).all()
    # an element is at most half a code step off: 1 above magnitude 4, in units of the scale
    assert (np.abs(q - v).reshape(50, 2, 32) <= s[..., None]).all()
    # requantising the values changes nothing
    assert (oracle.quantize_mxfp4(q)[2] == q).all()


def test_blocks_that_are_zero_tiny_or_not_finite():
    v = np.zeros((5, 32))
    v[1, 3] = 2.0 ** -149                    # below every scale: rounds to 0 at 2^-127
    v[2, 0] = np.inf
    v[3, 31] = np.nan
    v[4, 0] = float(np.finfo(np.float32).max)
    codes, sb, q = oracle.quantize_mxfp4(v)
    assert sb[:, 0].tolist() == [0, 0, 255, 255, 253]
    assert (codes[:4] == 0).all() and (q[:2] == 0).all() and np.isnan(q[2:4]).all()
    assert codes[4, 0] == 6 and (codes[4, 1:] == 0).all()    # fp32's largest, 4 * 2^126 below a tie


# ------------------------------------------------------------------ refusals

@pytest.mark.parametrize("d,cs,ss", [(128, 128, 16), (256, 128, 16), (384, 256, 16), (640, 384, 32),
                                     (4096, 2048, 128), (7168, 3584, 224)])
def test_row_strides(d, cs, ss):
    assert moe.mxfp4_strides(d) == (cs, ss)


@pytest.mark.parametrize("d", [0, -128, 96, 130])
def test_row_strides_refuse(d):
    with pytest.raises(moe.MoEError):
        moe.mxfp4_strides(d)


@pytest.mark.parametrize("kw,ok", [({}, True), ({"I": 64}, False), ({"I": 192}, False), ({"d": 192}, False),
                                   ({"activation": moe.MOE_ACT_RELU2}, True), ({"k": 9}, False)])
def test_packed_size(kw, ok):
    p = _p(**kw)
    assert (moe.packed_mxfp4_size(p) > 0) == ok
    if ok:
        gr = 2 if p.activation == moe.MOE_ACT_SWIGLU else 1
        up = lambda n: -(-n // 1024) * 1024
        want = up(128 * 256 * 2)                              # router, 128 padded rows
        want += up(8 * gr * 128 * 256 // 2) + up(8 * (gr * 128 // 64) * 1024)
        want += up(8 * 256 * 128 // 2) + up(8 * (256 // 64) * 1024)
        assert moe.packed_mxfp4_size(p) == want


def test_conversion_entries_refuse_before_launch():
    L = moe.lib()
    p = ctypes.byref(_p())
    bad = moe.MOE_ERR_INVALID_ARG
    assert L.moe_quantize_mxfp4(p, None, FAKE, FAKE, None) == bad
    assert L.moe_quantize_mxfp4(p, FAKE, None, FAKE, None) == bad
    assert L.moe_quantize_mxfp4(p, FAKE, FAKE, None, None) == bad
    assert L.moe_quantize_mxfp4(p, ODD, FAKE, FAKE, None) == bad
    assert L.moe_quantize_mxfp4(None, FAKE, FAKE, FAKE, None) == bad
    assert L.moe_dequantize_mxfp4(p, FAKE, FAKE, ODD, None) == bad
    assert L.moe_dequantize_mxfp4(p, FAKE, None, FAKE, None) == bad
    assert L.moe_pack_weights_mxfp4(p, FAKE, FAKE, None, FAKE, FAKE, None) == bad      # W3 missing
    assert L.moe_pack_weights_mxfp4(p, FAKE, FAKE, FAKE, ODD, FAKE, None) == bad
    assert L.moe_unpack_weights_mxfp4(p, FAKE, FAKE, None, FAKE, None) == bad
    r2 = ctypes.byref(_p(activation=moe.MOE_ACT_RELU2))
    assert L.moe_unpack_weights_mxfp4(r2, FAKE, FAKE, FAKE, FAKE, None) == bad         # no W3 in this layer
    u = ctypes.byref(_p(I=64))
    assert L.moe_pack_weights_mxfp4(u, FAKE, FAKE, FAKE, FAKE, FAKE, None) == moe.MOE_ERR_UNSUPPORTED
    assert L.moe_unpack_weights_mxfp4(u, FAKE, FAKE, FAKE, FAKE, None) == moe.MOE_ERR_UNSUPPORTED


def test_binding_refuses_tensors_the_kernels_would_misread():
    p = _p()
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="not on the current GPU"):
        moe.quantize_mxfp4(p, x)
    with pytest.raises(ValueError, match="expected"):
        moe.quantize_mxfp4(p, x.float())
    with pytest.raises(ValueError, match="expected"):
        moe.quantize_mxfp4(p, x[:3])
    with pytest.raises(ValueError, match="expected"):
        moe.dequantize_mxfp4(p, torch.zeros(4, 127, dtype=torch.uint8), torch.zeros(4, 16, dtype=torch.uint8))
    with pytest.raises(ValueError, match="expected"):
        moe.pack_weights_mxfp4(p, torch.zeros(256, 7, dtype=torch.bfloat16), None, None, None)
    with pytest.raises(moe.MoEError):
        moe.unpack_weights_mxfp4(_p(I=192), torch.zeros(4, dtype=torch.uint8))
