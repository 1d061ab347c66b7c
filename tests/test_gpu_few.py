"""The whole layer for a few tokens against the composed path (moe.forward,
moe.forward_mxfp4), whose own parity with float64 other tests establish, over
both weight formats, types, activations, odd widths, shares and awkward rows.

Routing (idx, w, logits) is equal bit for bit.  The products are the same
numbers too, but the composed path rounds each pair's y to bf16 before the
weighted sum and forward_few does not, so with the composed path's own y an
output may differ by
  sum_j w_j * 2^-8 |y_j|            (the rounding of y, at most half a step),
  + 2^-8 |out| twice for a bf16 out (each side's own rounding),
  + (k + 1) 2^-24 sum_j w_j |y_j|   (the fp32 sums).
That is the whole tolerance; rows whose reference is NaN must be NaN, and rows
of tokens without a local pick exactly zero."""
import numpy as np
import pytest
import torch

from combine_wave_level_amd import moe

pytestmark = pytest.mark.gpu

DT = {"bf16": (moe.MOE_BF16, torch.bfloat16), "f32": (moe.MOE_F32, torch.float32)}
GATED, UNGATED = moe.MOE_ACT_SWIGLU, moe.MOE_ACT_RELU2


class Few:
    def __init__(self, T, d, I, E, k, E_local=None, e_begin=0, x="bf16", act=GATED, out="bf16", mx=False, seed=0,
                 skew=0.0):
        self.mx = mx
        E_local = E if E_local is None else E_local
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.p = moe.problem(T=T, d=d, I=I, E_global=E, k=k, E_local=E_local, e_begin=e_begin, experts_per_wave=1,
                             x_dtype=DT[x][0], out_dtype=DT[out][0], activation=act)
        mk = lambda *s: (torch.randn(*s, generator=g, device="cuda") * 0.02).bfloat16()
        Wg = (torch.randn(d, E, generator=g, device="cuda") * 0.02).to(DT[x][1])
        W1, W2 = mk(E_local, d, I), mk(E_local, I, d)
        W3 = mk(E_local, d, I) if act == GATED else None
        self.x = torch.randn(T, d, generator=g, device="cuda").to(DT[x][1])
        self.bias = (torch.arange(E, device="cuda").float() * -skew) if skew else None
        self.packed = (moe.pack_weights_mxfp4 if mx else moe.pack_weights)(self.p, Wg, W1, W3, W2)
        self.ws = moe.workspace(self.p)

    def few(self, **kw):
        return moe.forward_few(self.p, self.x, self.packed, self.ws, bias=self.bias, want_logits=True, mxfp4=self.mx, **kw)

    def composed(self):
        f = moe.forward_mxfp4 if self.mx else moe.forward
        return f(self.p, self.x, self.packed, moe.workspace(self.p), bias=self.bias, want_logits=True)

    def check(self):
        want = self.composed()
        self.ws.fill_(0xA5)      # nothing in the workspace needs a value before the call
        got = self.few(out=torch.full((self.p.T, self.p.d), float("nan"), dtype=want["out"].dtype, device="cuda"))
        torch.cuda.synchronize()
        for n in ("idx", "logits", "w"):
            a, b = got[n], want[n]
            same = (a == b) | ((a != a) & (b != b))
            assert bool(same.all()), (n, int((~same).sum()), a[~same][:5], b[~same][:5])
        a, b = got["out"].double(), want["out"].double()
        pos = want["disp"].pair_pos
        y = want["y"].double()[pos.clamp(min=0).long()].abs()                # [T, k, d]
        w = torch.where(pos >= 0, want["w"].double(), torch.zeros_like(want["w"].double()))
        size = torch.where(pos.unsqueeze(-1) >= 0, y * w.unsqueeze(-1), torch.zeros_like(y)).sum(1)
        tol = size * (2.0 ** -8 + (self.p.k + 1) * 2.0 ** -24)
        if want["out"].dtype == torch.bfloat16:
            tol = tol + (2 * 2.0 ** -8) * (b.abs() + tol)
        nan = b != b
        assert torch.equal(nan, a != a)
        over = ((a - b).abs() - tol)[~nan]
        assert over.numel() == 0 or float(over.max()) <= 0, float(over.max())
        return got


CASES = [  # T, d, I, E, k, E_local, e_begin
    (1, 128, 128, 1, 1, 1, 0), (1, 256, 128, 8, 2, 8, 0), (2, 384, 256, 3, 3, 3, 0), (3, 640, 384, 7, 5, 7, 0),
    (16, 256, 256, 4, 4, 4, 0), (15, 1152, 640, 33, 6, 33, 0), (8, 512, 512, 65, 8, 65, 0), (5, 768, 128, 200, 12, 40, 80),
    (13, 2048, 512, 128, 6, 32, 0), (16, 1024, 256, 256, 8, 256, 0), (16, 128, 128, 64, 64, 64, 0), (7, 256, 128, 16, 1, 1, 15),
    (1, 7168, 2048, 32, 8, 32, 0),
    (16, 2176, 640, 80, 8, 80, 0), (9, 2048, 1024, 64, 3, 64, 0),   # two row blocks a wavefront in MXFP4
]


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("case", CASES)
def test_equals_the_composed_path(case, mx):
    T, d, I, E, k, E_local, e_begin = case
    print(f"[case] few {case} mx={mx}", flush=True)
    Few(T, d, I, E, k, E_local, e_begin, mx=mx, seed=T + d).check()


def test_most_pairs_with_two_row_blocks_a_wavefront():
    """16 tokens of 64 picks in the wider MXFP4 tile: the largest y in LDS."""
    print("[case] few 1024 pairs", flush=True)
    Few(16, 1024, 1024, 64, 64, mx=True, seed=7).check()
    Few(16, 1024, 1024, 256, 64, 96, 96, mx=True, seed=8).check()


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("x,act,out", [("f32", GATED, "f32"), ("f32", UNGATED, "bf16"), ("bf16", UNGATED, "f32"),
                                       ("bf16", GATED, "f32")])
def test_types_and_activations(x, act, out, mx):
    print(f"[case] few {x} {act} {out} mx={mx}", flush=True)
    for T, d, I, E, k in ((1, 256, 128, 8, 2), (11, 384, 384, 20, 3)):
        Few(T, d, I, E, k, x=x, act=act, out=out, mx=mx, seed=d).check()


def test_narrow_intermediate_of_the_bf16_experts():
    """I of 64 and 192: the bf16 experts accept any multiple of 64."""
    print("[case] few I=64, 192", flush=True)
    for I in (64, 192):
        Few(4, 256, I, 6, 2, seed=I).check()


@pytest.mark.parametrize("mx", [False, True])
def test_skewed_picks_and_tokens_without_local_expert(mx):
    print(f"[case] few skew mx={mx}", flush=True)
    # a strong skew sends every token to the same experts (16 rows each)
    r = Few(16, 256, 128, 32, 2, skew=5.0, mx=mx).check()
    assert (r["idx"] == torch.tensor([0, 1], device="cuda")).all()
    # a share that no token reaches: zeros
    r = Few(16, 256, 128, 32, 2, E_local=4, e_begin=20, skew=5.0, mx=mx).check()
    assert (r["out"] == 0).all()


@pytest.mark.parametrize("mx", [False, True])
def test_rows_that_are_not_finite_stay_their_own(mx):
    print(f"[case] few nan mx={mx}", flush=True)
    L = Few(6, 256, 128, 8, 3, mx=mx)
    clean = {n: v.clone() for n, v in L.check().items()}
    L.x[1, 5] = float("nan")
    L.x[4, 200] = float("inf")
    got = L.check()
    for t in (0, 2, 3, 5):
        for n in ("idx", "w", "out"):   # the others' rows do not change by a bit
            assert torch.equal(got[n][t], clean[n][t])


@pytest.mark.parametrize("mx", [False, True])
def test_ties_go_to_the_lower_expert(mx):
    print(f"[case] few ties mx={mx}", flush=True)
    L = Few(4, 256, 128, 70, 5, mx=mx)
    L.x.zero_()
    r = L.check()
    assert (r["idx"] == torch.arange(5, device="cuda")).all() and (r["out"] == 0).all()


@pytest.mark.parametrize("mx", [False, True])
def test_batch_invariance(mx):
    """A token's row does not depend on the tokens beside it."""
    print(f"[case] few invariance mx={mx}", flush=True)
    L = Few(16, 512, 256, 24, 4, mx=mx)
    whole = L.check()
    for t in (0, 7, 15):
        one = moe.forward_few(L.p.replace(T=1), L.x[t:t + 1].contiguous(), L.packed, L.ws, mxfp4=mx)
        torch.cuda.synchronize()
        for n in ("idx", "w", "out"):
            assert torch.equal(one[n][0], whole[n][t])


@pytest.mark.parametrize("act", [GATED, UNGATED])
def test_batch_invariance_across_wavefront_tiles(act):
    """16 tokens run two row blocks a wavefront, one token runs one."""
    print(f"[case] few tiles act={act}", flush=True)
    L = Few(16, 2048, 1152, 64, 8, act=act, mx=True)
    whole = L.check()
    for t in (0, 9):
        one = moe.forward_few(L.p.replace(T=1), L.x[t:t + 1].contiguous(), L.packed, L.ws, mxfp4=True)
        torch.cuda.synchronize()
        for n in ("idx", "w", "out"):
            assert torch.equal(one[n][0], whole[n][t])


def _graph(step, outs):
    """Four replays, each over poisoned outputs and followed by an eager step
    on the same workspace, give the eager step's bits."""
    step()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    captured = outs()
    torch.cuda.synchronize()
    for rep in range(4):
        for o in captured:
            o.view(torch.uint8).fill_(0x7F)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for o, w in zip(captured, want):
            assert torch.equal(o, w), rep
        step()
        torch.cuda.synchronize()
        for o, w in zip(outs(), want):
            assert torch.equal(o, w), rep


@pytest.mark.parametrize("mx", [False, True])
def test_graph_replays(mx):
    print(f"[case] few graph mx={mx}", flush=True)
    L = Few(5, 512, 256, 16, 4, mx=mx)
    got = {}

    def step():
        got.update(moe.forward_few(L.p, L.x, L.packed, L.ws, mxfp4=mx))

    _graph(step, lambda: [got["idx"], got["w"], got["out"]])


@pytest.mark.parametrize("T", [7, 300])
def test_graph_replays_of_the_mxfp4_layer(T):
    """route, dispatch, quantise, expert FFN: the streaming and the wide tiles."""
    print(f"[case] mxfp4 graph T={T}", flush=True)
    L = Few(T, 512, 256, 3, 2, mx=True)
    got = {}

    def step():
        got.update(moe.forward_mxfp4(L.p, L.x, L.packed, L.ws))

    _graph(step, lambda: [got["idx"], got["w"], got["out"]])


def test_on_another_stream_and_twice_on_one_workspace():
    """The calls follow the current stream; a second call on the workspace in
    the same stream finds nothing of the first."""
    print("[case] few streams", flush=True)
    A, B = Few(3, 512, 256, 16, 4, seed=1), Few(16, 256, 128, 8, 2, mx=True, seed=2)
    ra, rb = A.check(), B.check()
    n = max(moe.workspace_size(A.p), moe.workspace_size(B.p))
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = []
        for _ in range(5):
            got.append((moe.forward_few(A.p, A.x, A.packed, ws), moe.forward_few(B.p, B.x, B.packed, ws, mxfp4=True)))
    torch.cuda.synchronize()
    for a, b in got:
        assert torch.equal(a["out"], ra["out"]) and torch.equal(b["out"], rb["out"])


def test_refused_tensors():
    L = Few(4, 256, 128, 8, 2)
    with pytest.raises(ValueError, match="not contiguous"):
        moe.forward_few(L.p, L.x.t().contiguous().t(), L.packed, L.ws)
    with pytest.raises(ValueError, match="packed"):
        moe.forward_few(L.p, L.x, L.packed, L.ws, mxfp4=True)      # the other format's buffer
    with pytest.raises(moe.MoEError) as e:
        moe.forward_few(L.p, L.x, L.packed, L.ws[:1024])
    assert e.value.status == moe.MOE_ERR_WORKSPACE
    with pytest.raises(moe.MoEError) as e:
        off = torch.empty(4 * 256 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(4, 256)
        moe.forward_few(L.p, off, L.packed, L.ws)
    assert e.value.status == moe.MOE_ERR_INVALID_ARG
    with pytest.raises(ValueError, match="bias"):
        moe.forward_few(L.p, L.x, L.packed, L.ws, bias=torch.zeros(8, dtype=torch.float64, device="cuda"))


def test_no_tokens_and_too_many():
    L = Few(0, 256, 128, 8, 2)
    assert L.few()["out"].shape == (0, 256)
    L = Few(17, 256, 128, 8, 2)
    with pytest.raises(moe.MoEError) as e:
        L.few()
    assert e.value.status == moe.MOE_ERR_UNSUPPORTED
