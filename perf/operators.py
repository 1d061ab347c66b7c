"""Cases of the 4-bit and the few-token operators of the MoE layer share.

Four operators, by the case's "op":

  quant   a batch of token rows to MXFP4 (blocks of 32 along a row, one
          power-of-two scale a block) and back to the values the codes stand
          for (quantize_mxfp4, dequantize_mxfp4);
  pack    one layer's expert weights to MXFP4 along each product's reduction
          index, in the layout the products read, and back
          (pack_weights_mxfp4, unpack_weights_mxfp4);
  ffn     the expert FFN of a routed batch with both operands of both
          products in MXFP4, from bf16 or fp32 token rows to the combined
          output (quantize_mxfp4, ffn_mxfp4);
  few     the whole layer for at most 16 tokens, from token rows to routing
          and output, with bf16 or MXFP4 expert weights (forward_few).

``own`` selects what ``run`` computes with: the framework's operators where
it is true, their plain form in torch where it is false.  Weights of the
MXFP4 products are values of the 4-bit grid, as a checkpoint in that format
holds them, so that both forms multiply the same numbers.
"""
import math

import torch

own = False

BLOCK = 32


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a prefill batch of a d = 4096 layer on its way into 4-bit products
        dict(name="quant_prefill", op="quant", T=8192, d=4096, x="bf16"),
        # a decode step's rows, where the two launches are the cost; a width that is no power of two
        dict(name="quant_decode", op="quant", T=8, d=7168, x="f32"),
        # a layer's weights as they change while training with 4-bit weights
        dict(name="pack_layer", op="pack", E=16, d=4096, I=1024, w="bf16", act="swiglu"),
        # a narrow ungated layer of odd widths, master weights in fp32
        dict(name="pack_odd", op="pack", E=5, d=1152, I=640, w="f32", act="relu2"),
        # a training or prefill batch: the products' rate counts
        dict(name="ffn_batch", op="ffn", T=4096, d=4096, I=1024, E=16, E_local=16, k=4, zipf=0.0, x="bf16",
             act="swiglu"),
        # one GPU's share of an expert-parallel layer: about 256 rows an expert
        dict(name="ffn_share", op="ffn", T=8192, d=7168, I=2048, E=256, E_local=32, k=8, zipf=0.0, x="bf16",
             act="swiglu"),
        # a serving batch: every expert's weights for a few dozen rows
        dict(name="ffn_serve", op="ffn", T=128, d=7168, I=2048, E=32, E_local=32, k=8, zipf=1.2, x="bf16",
             act="swiglu"),
        # a small odd batch through ungated experts of odd widths
        dict(name="ffn_odd", op="ffn", T=37, d=1152, I=640, E=12, E_local=12, k=3, zipf=1.0, x="f32", act="relu2"),
        # one token of a large layer, the decode step of a single user
        dict(name="few_one", op="few", T=1, d=7168, I=2048, E=32, E_local=32, k=8, zipf=1.2, x="bf16", act="swiglu",
             weights="bf16"),
        # one token of a small layer, where latency is nearly all
        dict(name="few_one_small", op="few", T=1, d=2048, I=768, E=64, E_local=64, k=8, zipf=0.5, x="bf16",
             act="swiglu", weights="bf16"),
        # a decode step of eight users, experts in 4 bits
        dict(name="few_eight_mx", op="few", T=8, d=7168, I=2048, E=32, E_local=32, k=8, zipf=1.2, x="bf16",
             act="swiglu", weights="mxfp4"),
        # a share of a wide layer, an odd number of tokens, experts in 4 bits
        dict(name="few_share_mx", op="few", T=13, d=2048, I=512, E=128, E_local=32, k=6, zipf=0.5, x="bf16",
             act="swiglu", weights="mxfp4"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quant", "pack", "ffn", "ffn", "few", "few"))
    if op == "quant":
        return dict(op=op, T=_log(rng, 1, 8192), d=128 * _log(rng, 1, 56), x=rng.choice(("bf16", "f32")))
    act = rng.choice(("swiglu", "swiglu", "relu2"))
    if op == "pack":
        return dict(op=op, E=rng.randint(1, 16), d=128 * _log(rng, 2, 32), I=128 * _log(rng, 1, 16),
                    w=rng.choice(("bf16", "f32")), act=act)
    E_local = rng.randint(4, 32)
    E = min(256, E_local * rng.choice((1, 1, 2, 8)))
    c = dict(op=op, d=128 * _log(rng, 4, 56), I=128 * _log(rng, 4, 16), E=E, E_local=E_local, k=rng.randint(1, min(8, E)),
             zipf=rng.choice((0.0, 0.5, 1.2)), x=rng.choice(("bf16", "bf16", "f32")), act=act)
    if op == "few":
        return dict(c, T=rng.randint(1, 16), weights=rng.choice(("bf16", "mxfp4")))
    # at most the share's products
    pairs_a_token = max(1.0, c["k"] * E_local / E)
    most = int(8192 * 7168 * 2048 / (pairs_a_token * c["d"] * c["I"]))
    return dict(c, T=_log(rng, 1, max(1, min(8192, most))))


# ------------------------------------------------------------------ inputs

_DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


def _randn(g, shape, std, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _weights(g, shape, dtype, on_grid):
    """Expert matrices [E, K, N] ~ N(0, 0.02), one expert at a time."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    for e in range(shape[0]):
        w = _randn(g, shape[1:], 0.02, dtype)
        out[e] = (_to_grid(w.t()).t() if on_grid else w).to(dtype)
    return out


def _rows(g, T, d, dtype):
    """Token rows: N(0, 1) with a few channels far above the rest, as a
    layer's input has after its norm."""
    x = torch.randn((T, d), generator=g, device="cuda", dtype=torch.float32)
    far = torch.randint(0, d, (max(1, d // 256),), generator=g, device="cuda")
    x[:, far] *= 8.0
    return x.to(dtype)


def _plan(idx, E_local):
    """Rows of each local expert, padded to the longest: token of each slot
    [E_local, C], and the slot of each pair [T, k] (-1: expert not local)."""
    T, k = idx.shape
    flat = idx.reshape(-1).long()
    local = flat < E_local
    key = torch.where(local, flat, torch.full_like(flat, E_local))
    order = torch.sort(key, stable=True).indices
    counts = torch.bincount(key, minlength=E_local + 1)
    start = torch.cumsum(counts, 0) - counts
    rank = torch.empty_like(order)
    rank[order] = torch.arange(T * k, device=idx.device) - start[key[order]]
    C = max(1, int(counts[:E_local].max()))
    slot = torch.where(local, key * C + rank, torch.full_like(key, -1))
    rows = torch.zeros(E_local * C, dtype=torch.long, device=idx.device)
    rows[slot[local]] = (torch.arange(T * k, device=idx.device) // k)[local]
    return rows.reshape(E_local, C), slot.reshape(T, k)


def _problem(c, T):
    from combine_wave_level_amd import moe

    dt = {"bf16": moe.MOE_BF16, "f32": moe.MOE_F32}
    return moe.problem(T=T, d=c["d"], I=c.get("I", 128), E_global=c.get("E", 1), k=c.get("k", 1),
                       E_local=c.get("E_local", c.get("E", 1)), experts_per_wave=1, x_dtype=dt[c.get("x", "bf16")],
                       w_dtype=dt[c.get("w", "bf16")], out_dtype=moe.MOE_BF16,
                       activation=moe.MOE_ACT_RELU2 if c.get("act") == "relu2" else moe.MOE_ACT_SWIGLU)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    if c["op"] == "quant":
        s["x"] = _rows(g, c["T"], c["d"], _DTYPE[c["x"]])
        if own:
            s["p"] = _problem(c, c["T"])
        return s
    d, I = c["d"], c["I"]
    E_local = c.get("E_local", c.get("E"))
    grid = c["op"] == "ffn" or c.get("weights") == "mxfp4"
    wt = _DTYPE[c.get("w", "bf16")]
    s["W1"] = _weights(g, (E_local, d, I), wt, grid)
    s["W3"] = _weights(g, (E_local, d, I), wt, grid) if c["act"] == "swiglu" else None
    s["W2"] = _weights(g, (E_local, I, d), wt, grid)
    if c["op"] == "pack":
        s["Wg"] = _randn(g, (d, c["E"]), 0.02, torch.bfloat16)
        if own:
            s["p"] = _problem(c, 1)
        return s
    T, E, k = c["T"], c["E"], c["k"]
    s["x"] = _rows(g, T, d, _DTYPE[c["x"]])
    s["Wg"] = _randn(g, (d, E), 0.02, _DTYPE[c["x"]])
    # popularity of an expert falls as its rank to the power of -zipf
    rank = torch.randperm(E, generator=g, device="cuda").add(1).double()
    s["bias"] = (-c["zipf"] * rank.log()).float()
    if c["op"] == "ffn":
        u = torch.rand((T, E), generator=g, device="cuda", dtype=torch.float64)
        score = s["bias"].double() - (-u.log()).log()
        top, idx = torch.topk(score, k, dim=1)
        s["idx"], s["w"] = idx.int().contiguous(), torch.softmax(top, 1).float().contiguous()
        s["rows"], s["slot"] = _plan(s["idx"], E_local)
    if own:
        from combine_wave_level_amd import moe

        s["p"] = p = _problem(c, T)
        pack = moe.pack_weights_mxfp4 if grid else moe.pack_weights
        s["packed"] = pack(p, s["Wg"], s["W1"], s["W3"], s["W2"])
        s["ws"] = moe.workspace(p)
        if c["op"] == "ffn":
            s["disp"] = moe.dispatch(p, s["idx"], s["ws"])
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        return _run_own(s)
    c = s["case"]
    if c["op"] == "quant":
        return _to_grid(s["x"]).to(s["x"].dtype)
    if c["op"] == "pack":
        return {n: _to_grid(s[n].transpose(1, 2)).transpose(1, 2).to(s[n].dtype)
                for n in ("W1", "W3", "W2") if s[n] is not None}
    if c["op"] == "ffn":
        return _plain_ffn(s)
    return _plain_few(s)


def _run_own(s):
    from combine_wave_level_amd import moe

    c, p = s["case"], s["p"]
    if c["op"] == "quant":
        codes, scales = moe.quantize_mxfp4(p, s["x"])
        return moe.dequantize_mxfp4(p, codes, scales)
    if c["op"] == "pack":
        packed = moe.pack_weights_mxfp4(p, s["Wg"], s["W1"], s["W3"], s["W2"])
        W1, W3, W2 = moe.unpack_weights_mxfp4(p, packed)
        return {n: w for n, w in (("W1", W1), ("W3", W3), ("W2", W2)) if w is not None}
    if c["op"] == "ffn":
        codes, scales = moe.quantize_mxfp4(p, s["x"])
        return moe.ffn_mxfp4(p, codes, scales, s["packed"], s["disp"], s["w"], s["ws"])[1]
    r = moe.forward_few(p, s["x"], s["packed"], s["ws"], bias=s["bias"], mxfp4=c["weights"] == "mxfp4")
    return {"idx": r["idx"], "w": r["w"], "out": r["out"]}


def _to_grid(v):
    """MXFP4 values of v, blocks of 32 along the last axis, in fp32: scale 2^k
    with the smallest k >= -127 such that the block's largest magnitude is at
    most 6 * 2^k, elements to the nearest E2M1 value, ties to even."""
    b = v.float().unflatten(-1, (-1, BLOCK))
    f, e = torch.frexp(b.abs().amax(-1, keepdim=True))
    k = torch.where(f <= 0.75, e - 3, e - 2).clamp_(min=-127)
    # 2^-k as two factors inside fp32's range
    m = torch.ldexp(torch.ldexp(b.abs(), -torch.div(k, 2, rounding_mode="floor")),
                    torch.div(k, 2, rounding_mode="floor") - k)
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
    q = torch.round(m / step) * step
    half = torch.div(k, 2, rounding_mode="floor")
    return torch.copysign(torch.ldexp(torch.ldexp(q, half), k - half), b).flatten(-2)


def _activate(h1, h3):
    return torch.relu(h1).square() if h3 is None else h1 / (1 + torch.exp(-h1)) * h3


def _plain_ffn(s):
    x = _to_grid(s["x"])[s["rows"]]
    a = _activate(x @ s["W1"].float(), None if s["W3"] is None else x @ s["W3"].float())
    y = (_to_grid(a) @ s["W2"].float()).flatten(0, 1)
    w = torch.where(s["slot"] >= 0, s["w"], torch.zeros_like(s["w"]))
    return (y[s["slot"].clamp(min=0)] * w.unsqueeze(-1)).sum(1).to(torch.bfloat16)


def _plain_few(s):
    c, x = s["case"], s["x"].float()
    T, k, E_local = c["T"], c["k"], c["E_local"]
    logits = x @ s["Wg"].float() + s["bias"]
    top, idx = torch.sort(logits, dim=1, descending=True, stable=True)
    top, idx = top[:, :k], idx[:, :k]
    w = torch.exp(top - top[:, :1])
    w = w / w.sum(1, keepdim=True)
    mx = c["weights"] == "mxfp4"
    if mx:
        x = _to_grid(x)
    if T * k < E_local:
        # fewer picks than experts: the picked experts' weights, pair by pair
        at = idx.clamp(max=E_local - 1).flatten()
        rows = x.repeat_interleave(k, 0).unsqueeze(1)
    else:
        # every local expert on every token
        at = slice(None)
        rows = x.unsqueeze(0)
    a = _activate(rows @ s["W1"][at].float(), None if s["W3"] is None else rows @ s["W3"][at].float())
    y = (_to_grid(a) if mx else a) @ s["W2"][at].float()
    if T * k < E_local:
        y = y.reshape(T, k, -1)
    else:
        y = y[idx.clamp(max=E_local - 1), torch.arange(T, device=x.device).unsqueeze(1)]
    out = (y * torch.where(idx < E_local, w, torch.zeros_like(w)).unsqueeze(-1)).sum(1)
    return {"idx": idx.int(), "w": w, "out": out.to(torch.bfloat16)}


# ------------------------------------------------------------------ what a pass cannot do without

_BYTES = {"bf16": 2, "f32": 4}
_MX = 0.5 + 1 / BLOCK  # bytes of an MXFP4 element with its share of the scale


def work(case):
    c = dict(case)
    op = c["op"]
    if op == "quant":
        # x read, codes written and read, values written
        n = c["T"] * c["d"]
        return {"bytes": n * (2 * _BYTES[c["x"]] + 2 * _MX), "flops": 4 * n}
    mats = 3 if c["act"] == "swiglu" else 2
    one = mats * c["d"] * c["I"]  # weights of an expert
    if op == "pack":
        return {"bytes": c["E"] * one * (2 * _BYTES[c["w"]] + 2 * _MX), "flops": 4 * c["E"] * one}
    T, d, E, E_local, k = c["T"], c["d"], c["E"], c["E_local"], c["k"]
    share = E_local / E
    if op == "ffn":
        # experts that some token picks, each pick drawn by popularity
        touched, pairs, weight = _touched(c), T * k * share, _MX
        router = 0
    else:
        touched, pairs = _touched(c), T * k * share
        weight = _MX if c["weights"] == "mxfp4" else 2
        router = d * E * _BYTES[c["x"]]
    moved = touched * one * weight + router + T * d * (_BYTES[c["x"]] + 2)
    return {"bytes": moved, "flops": 2 * one * pairs + 2 * T * d * E * (op == "few")}


def _touched(c):
    """About how many local experts a batch picks: k distinct picks a token,
    each expert in proportion to its popularity where that leaves it below
    one pick a token."""
    p = [r ** -c["zipf"] for r in range(1, c["E"] + 1)]
    lo, hi = 0.0, c["k"] / min(p)
    for _ in range(60):
        mid = (lo + hi) / 2
        lo, hi = (mid, hi) if sum(min(1.0, mid * v) for v in p) < c["k"] else (lo, mid)
    hit = sum(1 - (1 - min(1.0, hi * v)) ** c["T"] for v in p)
    return max(1.0, hit * c["E_local"] / c["E"])


# ------------------------------------------------------------------ the definition in 64 bits

_MIDS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)
_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _mx64(v):
    """MXFP4 of a float64 tensor along the last axis: the code is the number
    of midpoints that lie below the scaled magnitude (at a tie, the even code)."""
    v = v.reshape(*v.shape[:-1], -1, BLOCK)
    big = v.abs().max(-1, keepdim=True).values
    k = torch.ceil(torch.log2(torch.where(big > 0, big, torch.ones_like(big)) / 6.0))
    k = torch.where(big > 0, k, torch.full_like(k, -127.0)).clamp(min=-127.0)
    scale = torch.pow(torch.full_like(k, 2.0), k)
    m = (v / scale).abs()
    code = torch.zeros_like(m, dtype=torch.long)
    for i, mid in enumerate(_MIDS):
        code += (m > mid) if i % 2 == 0 else (m >= mid)
    q = torch.tensor(_VALUES, dtype=torch.float64, device=v.device)[code] * scale
    q = torch.where(torch.signbit(v), -q, q)
    return q.reshape(*v.shape[:-2], -1)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "quant":
        return _mx64(s["x"].double())
    if c["op"] == "pack":
        out = {}
        for n in ("W1", "W3", "W2"):
            if s[n] is not None:
                out[n] = torch.stack([_mx64(w.double().t()).t() for w in s[n]])
        return out
    few = c["op"] == "few"
    x = s["x"].double()
    res = {}
    if few:
        logits = x @ s["Wg"].double() + s["bias"].double()
        prob = torch.softmax(logits, 1)
        order = torch.argsort(-logits, dim=1, stable=True)[:, : c["k"]]
        w = prob.gather(1, order)
        w = w / w.sum(1, keepdim=True)
        idx = order
        res = {"idx": idx.int(), "w": w}
    else:
        idx, w = s["idx"].long(), s["w"].double()
    mx = not few or c["weights"] == "mxfp4"
    if mx:
        x = _mx64(x)
    out = torch.zeros((c["T"], c["d"]), dtype=torch.float64, device=x.device)
    for e in range(c["E_local"]):
        t, j = torch.nonzero(idx == e, as_tuple=True)
        if not t.numel():
            continue
        h = x[t] @ s["W1"][e].double()
        a = torch.clamp(h, min=0) ** 2 if s["W3"] is None else h * torch.sigmoid(h) * (x[t] @ s["W3"][e].double())
        if mx:
            a = _mx64(a)
        out.index_add_(0, t, (a @ s["W2"][e].double()) * w[t, j].unsqueeze(1))
    return dict(res, out=out) if few else out
