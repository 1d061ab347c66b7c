"""MXFP4 conversions on the GPU, through the C ABI: codes, scales and values
equal the float64 oracle's bit for bit (no rounding is left to tolerate: a
code is a choice among eight values and a value times a power of two is
exact)."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from combine_wave_level_amd import moe

pytestmark = pytest.mark.gpu

GATED, UNGATED = moe.MOE_ACT_SWIGLU, moe.MOE_ACT_RELU2
DT = {"bf16": (moe.MOE_BF16, torch.bfloat16), "f32": (moe.MOE_F32, torch.float32)}


def _problem(T=1, d=256, I=128, E=1, x="bf16", w="bf16", act=moe.MOE_ACT_SWIGLU):
    return moe.problem(T=T, d=d, I=I, E_global=E, k=1, experts_per_wave=1, x_dtype=DT[x][0], w_dtype=DT[w][0],
                       activation=act)


def _unpack_codes(c, d):
    return np.stack([c & 15, c >> 4], -1).reshape(c.shape[0], -1)[:, :d], c[:, d // 2:]


def _same(a, b):
    bad = np.argwhere(~((a == b) | (np.isnan(a) & np.isnan(b))))
    for i in bad[:5]:
        print("  differs at", tuple(i), a[tuple(i)], b[tuple(i)], flush=True)
    return len(bad) == 0


def _check_rows(x, dt):
    """x: float32 array whose values the type holds."""
    T, d = x.shape
    p = _problem(T=T, d=d, x=dt)
    xd = torch.from_numpy(x).cuda().to(DT[dt][1])
    x64 = xd.cpu().float().numpy().astype(np.float64)
    codes, scales = moe.quantize_mxfp4(p, xd)
    back = moe.dequantize_mxfp4(p, codes, scales)
    torch.cuda.synchronize()
    assert back.dtype == xd.dtype
    oc, osb, ov = oracle.quantize_mxfp4(x64)
    got, pad = _unpack_codes(codes.cpu().numpy(), d)
    sb = scales.cpu().numpy()
    assert (sb[:, :d // 32] == osb).all() and (sb[:, d // 32:] == 0).all() and (pad == 0).all()
    assert (got == oc).all()
    # the value in the type: exact, but 4 * 2^126 = 2^128 (a block of fp32's
    # last half binade rounds up to it) lies half a step above the largest
    # fp32, 2^128 - 2^104, and is infinity there
    with np.errstate(over="ignore"):
        ov = ov.astype(np.float32).astype(np.float64)
    assert _same(back.cpu().float().numpy().astype(np.float64), ov)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", [(1, 128), (3, 256), (2, 384), (17, 640), (5, 1152), (301, 4096), (8, 7168)])
def test_rows(T, d, dt):
    print(f"[case] mxfp4 rows T={T} d={d} {dt}", flush=True)
    rng = np.random.default_rng(T * d)
    x = rng.standard_normal((T, d)) * np.exp2(rng.integers(-20, 20, (T, 1)))
    _check_rows(x.astype(np.float32), dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_crafted_blocks(dt):
    print(f"[case] mxfp4 crafted {dt}", flush=True)
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    x = np.zeros((9, 256), dtype=np.float64)
    x[0, :7], x[0, 8:15], x[0, 16] = mids, -mids, 6.0                       # ties
    step = 2.0 ** (-7 if dt == "bf16" else -20)
    x[0, 32:39], x[0, 40:47], x[0, 48] = mids * (1 + step), -mids * (1 - step), -6.0   # just past them
    x[1, 0:32] = -1e-9                                                      # one value fills a block
    x[1, 32], x[1, 33] = -6.0, -0.2                                         # rounds to -0
    x[2, :3] = [6.0 * 2.0 ** 5, 1, 2]                                       # amax on the border
    x[2, 32:35] = [6.0 * 2.0 ** 5 * (1 + 2.0 ** -7), 1, 2]                  # and just above
    x[3, 0], x[3, 32], x[3, 64] = 2.0 ** -126, 2.0 ** -127, 1.5 * 2.0 ** -124   # the smallest scales
    x[4, 0], x[4, 33] = np.float32(3.0e38), np.float32(-2.0e38)             # the largest
    x[5, 5], x[5, 40], x[5, 70] = np.inf, -np.inf, np.nan                   # whole blocks read as NaN
    x[5, 6] = 3.0
    x[6] = np.linspace(-6, 6, 256)
    x[7, 96:128] = np.arange(32) * 2.0 ** -120
    _check_rows(x.astype(np.float32), dt)


def test_rows_past_two_to_the_35_elements():
    """More elements than one launch has threads for: the rows at both ends
    and around the border between launches are those of a small call."""
    T, d = (1 << 24) - 3, 2176
    if torch.cuda.mem_get_info()[0] < 130 << 30:
        pytest.skip("needs 130 GiB of free memory")
    print(f"[case] mxfp4 rows T={T} d={d}", flush=True)
    p, border = _problem(T=T, d=d), (1 << 34) // d
    at = torch.tensor([0, 1, border - 1, border, border + 1, T - 2, T - 1], device="cuda")
    rows = torch.randn(len(at), d, generator=torch.Generator("cuda").manual_seed(5), device="cuda").bfloat16()
    x = torch.zeros(T, d, dtype=torch.bfloat16, device="cuda")
    x[at] = rows
    codes, scales = moe.quantize_mxfp4(p, x)
    del x
    small = p.replace(T=len(at))
    c, s = moe.quantize_mxfp4(small, rows)
    assert torch.equal(codes[at], c) and torch.equal(scales[at], s)
    back = moe.dequantize_mxfp4(p, codes, scales)
    assert torch.equal(back[at], moe.dequantize_mxfp4(small, c, s))
    rest = torch.tensor([2, border // 2, border + 2, T - 3], device="cuda")
    assert not back[rest].any() and not codes[rest].any()
    del back, codes, scales
    torch.cuda.empty_cache()


def test_no_rows():
    p = _problem(T=0)
    codes, scales = moe.quantize_mxfp4(p, torch.empty(0, 256, dtype=torch.bfloat16, device="cuda"))
    assert moe.dequantize_mxfp4(p, codes, scales).shape == (0, 256)


@pytest.mark.parametrize("E,d,I,w,act", [(1, 128, 128, "bf16", moe.MOE_ACT_SWIGLU), (3, 384, 256, "f32", moe.MOE_ACT_SWIGLU),
                                         (2, 640, 384, "bf16", moe.MOE_ACT_RELU2), (2, 1152, 640, "f32", moe.MOE_ACT_RELU2),
                                         (2, 512, 1024, "bf16", moe.MOE_ACT_SWIGLU)])
def test_weights_round_trip(E, d, I, w, act):
    """pack then unpack equals the oracle's values of blocks along d (W1, W3)
    and along I (W2)."""
    print(f"[case] mxfp4 weights E={E} d={d} I={I} {w} act={act}", flush=True)
    g = torch.Generator().manual_seed(E * d + I)
    mk = lambda *s: (torch.randn(*s, generator=g) * 0.02).to(DT[w][1])
    W1, W2 = mk(E, d, I), mk(E, I, d)
    W3 = mk(E, d, I) if act == moe.MOE_ACT_SWIGLU else None
    W1[0, :32, 0] = 0
    W1[E - 1, 5, I - 1] = float("nan")
    p = _problem(d=d, I=I, E=E, w=w, act=act)
    Wg = torch.zeros(d, E, dtype=torch.bfloat16, device="cuda")
    D1, D3, D2 = W1.cuda(), None if W3 is None else W3.cuda(), W2.cuda()
    packed = moe.pack_weights_mxfp4(p, Wg, D1, D3, D2)
    # every byte is written: the same again over a poisoned buffer
    again = torch.full_like(packed, 0xA5)
    st = moe.lib().moe_pack_weights_mxfp4(ctypes.byref(p), moe._p(Wg), moe._p(D1), moe._p(D3), moe._p(D2),
                                          moe._p(again), moe._stream())
    assert st == moe.MOE_OK
    got = moe.unpack_weights_mxfp4(p, packed)
    torch.cuda.synchronize()
    gr = 1 if W3 is None else 2
    for off, n in _regions(p, gr):
        assert torch.equal(packed[off:off + n], again[off:off + n])
    for name, src, out in (("W1", W1, got[0]), ("W3", W3, got[1]), ("W2", W2, got[2])):
        if src is None:
            assert out is None
            continue
        assert out.dtype == src.dtype and out.shape == src.shape
        want = oracle.quantize_mxfp4(np.swapaxes(src.double().numpy(), 1, 2))[2]
        assert _same(np.swapaxes(out.float().cpu().numpy().astype(np.float64), 1, 2), want), name


def _regions(p, gr):
    """(offset, bytes) of the parts of the packed buffer."""
    up = lambda n: -(-n // 1024) * 1024
    off, out = 0, []
    kq = lambda K: -(-K // 512)
    for n in (128 * p.d * 2, p.E_local * gr * p.I * p.d // 2, p.E_local * (gr * p.I // 64) * kq(p.d) * 1024,
              p.E_local * p.d * p.I // 2, p.E_local * (p.d // 64) * kq(p.I) * 1024):
        out.append((off, n))
        off += up(n)
    assert off == moe.packed_mxfp4_size(p)
    return out


def test_the_packed_buffer_routes_like_the_bf16_one():
    p = _problem(T=33, d=512, I=256, E=8)
    p = p.replace(k=3)
    g = torch.Generator().manual_seed(1)
    mk = lambda *s: (torch.randn(*s, generator=g) * 0.02).bfloat16().cuda()
    Wg, W1, W3, W2, x = mk(512, 8), mk(8, 512, 256), mk(8, 512, 256), mk(8, 256, 512), mk(33, 512)
    ws = moe.workspace(p)
    a = moe.route(p, x, moe.pack_weights(p, Wg, W1, W3, W2), ws, want_logits=True)
    b = moe.route(p, x, moe.pack_weights_mxfp4(p, Wg, W1, W3, W2), ws, want_logits=True)
    torch.cuda.synchronize()
    for u, v in zip(a, b):
        assert torch.equal(u, v)


def test_refused_tensors():
    p = _problem(T=4)
    wide = torch.zeros(4, 512, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="not contiguous"):
        moe.quantize_mxfp4(p, wide[:, :256])
    with pytest.raises(ValueError, match="not contiguous"):
        moe.quantize_mxfp4(p, torch.zeros(256, 4, dtype=torch.bfloat16, device="cuda").t())
    # a row slice that starts off 16 bytes
    with pytest.raises(moe.MoEError):
        moe.quantize_mxfp4(p, torch.zeros(4 * 256 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(4, 256))


# ------------------------------------------------------------------ the expert FFN

def _layer(T, d, I, E, k, E_local=None, x="bf16", act=moe.MOE_ACT_SWIGLU, out=moe.MOE_BF16, seed=0, e_begin=0):
    """Seeded weights and rows on the device, packed, with the float64 values
    that the 4-bit operands stand for."""
    E_local = E if E_local is None else E_local
    g = torch.Generator().manual_seed(seed)
    p = moe.problem(T=T, d=d, I=I, E_global=E, k=k, E_local=E_local, e_begin=e_begin, experts_per_wave=1,
                    x_dtype=DT[x][0], out_dtype=out, activation=act)
    mk = lambda *s: (torch.randn(*s, generator=g) * 0.02).bfloat16()
    W1, W2 = mk(E_local, d, I), mk(E_local, I, d)
    W3 = mk(E_local, d, I) if act == moe.MOE_ACT_SWIGLU else None
    Wg = (torch.randn(d, E, generator=g) * 0.02).to(DT[x][1])
    xr = torch.randn(T, d, generator=g).to(DT[x][1])
    L = dict(p=p, W1=W1, W3=W3, W2=W2, Wg=Wg.cuda(), x=xr.cuda(), g=g, xr=xr)
    L["packed"] = moe.pack_weights_mxfp4(p, L["Wg"], W1.cuda(), None if W3 is None else W3.cuda(), W2.cuda())
    L["ws"] = moe.workspace(p)
    return L


def _grid(a, axis=-1):
    a = np.swapaxes(a.double().numpy() if isinstance(a, torch.Tensor) else a, axis, -1)
    return np.swapaxes(oracle.quantize_mxfp4(a)[2], axis, -1)


def _routing(L, idx, w):
    """Dispatch and MXFP4 rows of a routing given on the host."""
    idx_d = torch.as_tensor(idx, dtype=torch.int32).cuda()
    w_d = torch.as_tensor(w, dtype=torch.float32).cuda()
    disp = moe.dispatch(L["p"], idx_d, L["ws"])
    return disp, w_d


def _reference(L, idx, w, toks):
    """out of tokens toks in float64, a quantised in float64; and a bound of
    what a flipped code of a can change.

    The kernel's a differs from the float64 one by fp32 rounding, so an
    element next to a rounding border (or a block next to a scale border) can
    land on the other side: its value then moves by one code step, at most a
    third of itself plus a quarter of the block's scale.  `flip` is what one
    flip of the largest element of each row times its largest weight can move
    an output by."""
    p = L["p"]
    x = _grid(L["xr"][toks])
    W1, W2 = _grid(L["W1"], 1), _grid(L["W2"], 1)
    W3 = None if L["W3"] is None else _grid(L["W3"], 1)
    out = np.zeros((len(toks), p.d))
    flip = np.zeros(len(toks))
    for i, t in enumerate(toks):
        for j in range(p.k):
            e = int(idx[t, j]) - p.e_begin
            if not 0 <= e < p.E_local:
                continue
            h1 = x[i] @ W1[e]
            a = np.maximum(h1, 0) ** 2 if W3 is None else h1 / (1 + np.exp(-h1)) * (x[i] @ W3[e])
            aq = _grid(a)
            out[i] += w[t, j] * (aq @ W2[e])
            flip[i] += w[t, j] * np.abs(aq).max() / 3 * np.abs(W2[e]).max()
    return out, flip


def _check_out(L, idx, w, out, toks):
    """|out - ref| per element: y's rounding to bf16 (2^-8 of each |y|, so at
    most 2^-8 of sum_j w_j |y_j|), out's own (2^-8 of |out|), fp32 sums (far
    below), and at most two flipped codes of a row."""
    ref, flip = _reference(L, idx, w, toks)
    got = out[toks].float().cpu().numpy().astype(np.float64)
    tol = 2.0 ** -7 * np.abs(ref).max(1) * 1.5 + 2 * flip
    err = np.abs(got - ref).max(1)
    print(f"  max err {err.max():.3g} of {np.abs(ref).max():.3g}; rms {np.sqrt(((got - ref) ** 2).mean()):.3g} "
          f"of {np.sqrt((ref ** 2).mean()):.3g}", flush=True)
    assert (err <= tol).all(), (err - tol).max()
    # flips are rare: over all tokens the error is that of the two bf16 roundings
    assert np.sqrt(((got - ref) ** 2).mean()) <= 2.0 ** -8 * 2 * np.sqrt((ref ** 2).mean()) + 1e-30


def _random_routing(L, seed=1, skew=None):
    p = L["p"]
    rng = np.random.default_rng(seed)
    score = rng.random((p.T, p.E_global))
    if skew is not None:
        score += skew
    idx = np.argsort(-score, 1)[:, :p.k].astype(np.int32)
    w = rng.random((p.T, p.k)) + 0.1
    return idx, (w / w.sum(1, keepdims=True)).astype(np.float32)


FFN = [  # T, d, I, E, k, E_local, x, act
    (1, 128, 128, 1, 1, 1, "bf16", 0), (1, 256, 128, 4, 2, 4, "f32", 0), (5, 384, 256, 4, 3, 4, "bf16", 1),
    (16, 640, 384, 5, 5, 5, "bf16", 0), (37, 1152, 640, 12, 3, 12, "f32", 1), (64, 512, 512, 1, 1, 1, "bf16", 0),
    (65, 512, 256, 2, 2, 2, "bf16", 0),
    (200, 256, 256, 2, 1, 2, "bf16", 0),      # the wide tiles from here: 256 by 256
    (257, 384, 384, 2, 2, 2, "bf16", 1),      # 128 by 256, odd numbers of K steps
    (300, 128, 128, 1, 1, 1, "bf16", 0),      # a single K step
    (600, 640, 128, 3, 2, 3, "f32", 0),
    (513, 896, 640, 4, 4, 2, "bf16", 0),      # a share
    (1100, 1024, 512, 4, 2, 4, "bf16", 0),
    (100, 128, 128, 1, 1, 1, "bf16", 0),      # many rows, but y has no room for the gathered operand
    (130, 512, 256, 4, 2, 4, "bf16", 1), (128, 512, 256, 4, 2, 4, "bf16", 0),   # the border between the tiles
]


@pytest.mark.parametrize("T,d,I,E,k,E_local,x,act", FFN)
def test_ffn_against_float64(T, d, I, E, k, E_local, x, act):
    print(f"[case] mxfp4 ffn T={T} d={d} I={I} E={E}/{E_local} k={k} {x} act={act}", flush=True)
    L = _layer(T, d, I, E, k, E_local, x, act, seed=T + d)
    idx, w = _random_routing(L)
    disp, w_d = _routing(L, idx, w)
    codes, scales = moe.quantize_mxfp4(L["p"], L["x"])
    y, out = moe.ffn_mxfp4(L["p"], codes, scales, L["packed"], disp, w_d, L["ws"])
    torch.cuda.synchronize()
    moe.check_error(L["ws"])
    toks = np.arange(T) if T <= 64 else np.unique(np.r_[0, T - 1, np.random.default_rng(0).choice(T, 40)])
    _check_out(L, idx, w, out, toks)
    # the standalone combine of the same y
    assert torch.equal(moe.combine(L["p"], y, disp.pair_pos, w_d), out)


@pytest.mark.parametrize("d,I,act", [(512, 256, GATED), (640, 384, UNGATED), (256, 128, GATED)])
def test_a_token_is_the_same_in_any_batch(d, I, act):
    """T = 1, 40 (64-row tiles) and 700 (256-row tiles): the rows and outputs
    of the same tokens have the same bits."""
    print(f"[case] mxfp4 invariance d={d} I={I} act={act}", flush=True)
    L = _layer(700, d, I, 4, 2, act=act, seed=5)
    idx, w = _random_routing(L)
    outs = {}
    for T, toks in ((700, np.arange(700)), (40, np.arange(330, 370)), (1, np.array([350]))):
        p = L["p"].replace(T=T)
        ws = moe.workspace(p)
        x = L["x"][torch.as_tensor(toks).cuda()].contiguous()
        disp = moe.dispatch(p, torch.as_tensor(idx[toks]).cuda(), ws)
        codes, scales = moe.quantize_mxfp4(p, x)
        outs[T] = moe.ffn_mxfp4(p, codes, scales, L["packed"], disp, torch.as_tensor(w[toks]).cuda(), ws)[1]
    torch.cuda.synchronize()
    assert torch.equal(outs[40], outs[700][330:370])
    assert torch.equal(outs[1], outs[700][350:351])


def test_no_rows_and_no_local_rows():
    L = _layer(5, 256, 128, 8, 2, E_local=2, seed=3)
    p = L["p"]
    disp, w_d = _routing(L, np.tile([5, 7], (5, 1)), np.full((5, 2), 0.5))
    codes, scales = moe.quantize_mxfp4(p, L["x"])
    out = torch.full((5, 256), float("nan"), dtype=torch.bfloat16, device="cuda")
    moe.ffn_mxfp4(p, codes, scales, L["packed"], disp, w_d, L["ws"], out=out)
    assert (out == 0).all()
    q = p.replace(T=0)
    ws = moe.workspace(q)
    disp = moe.dispatch(q, torch.empty(0, 2, dtype=torch.int32, device="cuda"), ws)
    e = torch.empty(0, 128, dtype=torch.uint8, device="cuda")
    y, out = moe.ffn_mxfp4(q, e, e[:, :16].contiguous(), L["packed"], disp,
                           torch.empty(0, 2, device="cuda"), ws)
    assert out.shape == (0, 256)


def test_all_rows_on_one_expert():
    """Every token picks the same expert of many: more m-tiles than the mean suggests."""
    print("[case] mxfp4 ffn hot expert", flush=True)
    L = _layer(333, 512, 256, 16, 1, seed=9)
    idx, w = np.full((333, 1), 11, np.int32), np.ones((333, 1), np.float32)
    disp, w_d = _routing(L, idx, w)
    codes, scales = moe.quantize_mxfp4(L["p"], L["x"])
    out = moe.ffn_mxfp4(L["p"], codes, scales, L["packed"], disp, w_d, L["ws"])[1]
    torch.cuda.synchronize()
    _check_out(L, idx, w, out, np.r_[0, 63, 64, 127, 200, 332])


def test_rows_that_are_not_finite_stay_their_own():
    print("[case] mxfp4 ffn nan", flush=True)
    for T in (9, 300):
        L = _layer(T, 256, 128, 4, 2, seed=4)
        idx, w = _random_routing(L)
        disp, w_d = _routing(L, idx, w)

        def run():
            codes, scales = moe.quantize_mxfp4(L["p"], L["x"])
            return moe.ffn_mxfp4(L["p"], codes, scales, L["packed"], disp, w_d, L["ws"])[1].clone()

        clean = run()
        L["x"][3, 40] = float("nan")
        L["x"][7, 200] = float("inf")
        bad = run()
        torch.cuda.synchronize()
        keep = [t for t in range(T) if t not in (3, 7)]
        assert torch.equal(bad[keep], clean[keep])
        assert bool(torch.isnan(bad[3]).all()) and bool(torch.isnan(bad[7]).all())


def test_quantised_weights_through_the_bf16_path():
    """What a layer trained on the 4-bit weights runs: unpacked values, packed
    for bf16, give the float64 layer on those values within the bf16 path's
    row tolerance (2e-2), and its gradients are finite."""
    print("[case] mxfp4 weights, bf16 layer", flush=True)
    L = _layer(48, 256, 128, 4, 2, seed=6)
    p = L["p"]
    W1, W3, W2 = moe.unpack_weights_mxfp4(p, L["packed"])
    for got, src in ((W1, L["W1"]), (W3, L["W3"]), (W2, L["W2"])):
        assert _same(got.float().cpu().numpy().astype(np.float64), _grid(src, 1))
    packed, packed_bwd = moe.pack_weights(p, L["Wg"], W1, W3, W2), moe.pack_weights_bwd(p, L["Wg"], W1, W3, W2)
    ws = moe.workspace(p, backward=True)
    r = moe.forward(p, L["x"], packed, ws)
    g = moe.backward(p, L["x"], packed, packed_bwd, r["idx"], r["w"], r["disp"], r["out"], ws, want_dw=True)
    torch.cuda.synchronize()
    assert all(bool(torch.isfinite(g[n]).all()) for n in ("dx", "dWg", "dW1", "dW3", "dW2"))
    idx, w = r["idx"].cpu().numpy(), r["w"].cpu().numpy().astype(np.float64)
    ref = oracle.forward_tokens(L["xr"].double().numpy(), idx, w, _grid(L["W1"], 1), _grid(L["W3"], 1),
                                _grid(L["W2"], 1), 0, 4)
    err = np.abs(r["out"].float().cpu().numpy() - ref).max(1) / np.abs(ref).max(1)
    assert err.max() <= 2e-2
