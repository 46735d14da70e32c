"""Cases and plain forms of the expert routing operators and of the gated activation that keeps
an 8-bit checkpoint.

Four operators, as the package offers them:

- ``route``: (token, choice) entries sorted by expert, into segments padded to 32 rows.
- ``dispatch``, ``quantize_dispatch`` and ``quantize_dispatch_dual``: the tokens' rows copied into
  those segments, as they are or straight into the MXFP8 operands of the grouped GEMMs.
- ``combine`` and ``combine_backward``: the weighted sum of a token's rows, and the gradients with
  respect to the rows and the weights.
- ``swiglu`` and ``swiglu_backward``: h = silu(gate) * up with gate and up kept in MXFP8, and the
  gradient from that copy.

``own`` chooses between the plain form (elementary torch operations in 32 bits) and the
package's kernels. Sizes are those of the expert layer and of the dense layers that the package's
workloads name, and generic ones around them.
"""
import math

import torch

own = False

FP8_MAX = 448.0
HIDDEN, EXPERTS, CHOICES, EXPERT_WIDTH = 2048, 128, 8, 768   # the package's expert layer
DENSE_WIDTH = 12288                                          # its dense gate / up width
MOST_ROUTED = 8192 * CHOICES * HIDDEN                        # elements of the largest routed copy
MOST_GATED = 4096 * DENSE_WIDTH                              # and of the largest activation


# ------------------------------------------------------------------------------- cases

def _routed(what, tokens, k, experts, dropped=0.0, **more):
    return dict(what=what, tokens=tokens, k=k, experts=experts, dropped=dropped, **more)


def listed():
    return [
        # one token's choices while a sampler decodes
        dict(name="route_1", **_routed("route", 1, CHOICES, EXPERTS)),
        # a micro-batch's choices
        dict(name="route_8192", **_routed("route", 8192, CHOICES, EXPERTS)),
        # an odd number of packed tokens, some entries dropped over capacity, FP32 rows
        dict(name="dispatch_1021", **_routed("dispatch", 1021, 6, 64, 0.1, cols=1999,
                                             dtype="fp32", form="plain", weighted=True)),
        # a decode batch on its way into the experts' forward product
        dict(name="dispatch_quant_37", **_routed("dispatch", 37, CHOICES, EXPERTS, cols=HIDDEN,
                                                 dtype="bf16", form="row", weighted=False)),
        # a micro-batch on its way into the experts' forward product and weight gradient
        dict(name="dispatch_dual_8192", **_routed("dispatch", 8192, CHOICES, EXPERTS,
                                                  cols=HIDDEN, dtype="bf16", form="dual",
                                                  weighted=False)),
        # one token's expert results
        dict(name="combine_1", **_routed("combine", 1, CHOICES, EXPERTS, cols=HIDDEN,
                                         dtype="bf16", weighted=True)),
        # a micro-batch's expert results
        dict(name="combine_8192", **_routed("combine", 8192, CHOICES, EXPERTS, cols=HIDDEN,
                                            dtype="bf16", weighted=True)),
        # the gradient of a few sequences, FP32 rows of an odd width, some entries dropped
        dict(name="combine_grad_509", **_routed("combine_grad", 509, 4, 16, 0.1, cols=1033,
                                                dtype="fp32", weighted=True)),
        # the gradient of a micro-batch
        dict(name="combine_grad_8192", **_routed("combine_grad", 8192, CHOICES, EXPERTS,
                                                 cols=HIDDEN, dtype="bf16", weighted=True)),
        # a decode batch through a dense block: nothing is kept
        dict(name="swiglu_37", what="swiglu", rows=37, width=DENSE_WIDTH, keep=False,
             rule="ceil"),
        # a micro-batch through a dense block of a learner
        dict(name="swiglu_4096", what="swiglu", rows=4096, width=DENSE_WIDTH, keep=True,
             rule="ceil"),
        # its way back, with the activation for the next weight gradient
        dict(name="swiglu_grad_4096", what="swiglu_grad", rows=4096, width=DENSE_WIDTH,
             again=True, rule="ceil"),
    ]


def _size(rng, lo, hi, unit=1):
    """A multiple of `unit` between `unit * lo` and `unit * hi`, spread over its logarithm."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return unit * min(hi, max(lo, n))


def draw(rng):
    what = rng.choice(["route", "dispatch", "dispatch", "combine", "combine_grad", "swiglu",
                       "swiglu_grad"])
    if what.startswith("swiglu"):
        while True:
            rows, width = _size(rng, 1, 70000), _size(rng, 2, 512, 32)
            if rows * width <= MOST_GATED:
                break
        case = dict(what=what, rows=rows, width=width, rule=rng.choice(["ceil", "floor"]))
        case["keep" if what == "swiglu" else "again"] = rng.choice([True, True, False])
        return case
    k, experts = rng.choice([1, 2, 4, 6, 8]), rng.choice([8, 16, 60, 64, 128, 256])
    dropped = rng.choice([0.0, 0.0, 0.1, 0.5])
    if what == "route":
        return _routed(what, _size(rng, 1, 8192 * CHOICES // k), k, experts, dropped)
    form = rng.choice(["plain", "row", "col", "dual"]) if what == "dispatch" else "plain"
    dtype = "bf16" if form != "plain" else rng.choice(["bf16", "fp32"])
    while True:
        tokens = _size(rng, 1, 16384)
        cols = _size(rng, 64, 8192) if form == "plain" else _size(rng, 2, 256, 32)
        rows = _rows(tokens, k, experts)
        if rows * cols * (4 if dtype == "fp32" else 2) <= 2 * MOST_ROUTED:
            break
    weighted = True if what == "combine_grad" else rng.choice([True, False])
    return _routed(what, tokens, k, experts, dropped, cols=cols, dtype=dtype, form=form,
                   weighted=weighted)


def _rows(tokens, k, experts):
    """Rows that any choice of experts fits in: every expert in use pads to 32."""
    n = tokens * k
    return (n + 31 * min(experts, n)) // 32 * 32


# ----------------------------------------------------------------------- inputs of a case

def _choices(case, g):
    """[tokens, k] distinct experts a token, popular ones first (rank^-1.1), -1 where dropped."""
    t, k, e = case["tokens"], case["k"], case["experts"]
    rank = torch.randperm(e, generator=g, device="cuda") + 1
    u = torch.rand(t, e, generator=g, device="cuda").clamp(1e-12, 1 - 1e-7)
    score = -1.1 * rank.float().log() - (-u.log()).log()
    ids = score.topk(min(k, e), dim=1).indices
    if case["dropped"]:
        gone = torch.rand(ids.shape, generator=g, device="cuda") < case["dropped"]
        ids = torch.where(gone, -1, ids)
    return ids


def _activations(rows, cols, g):
    """N(0, 1) with a few outlier features, in BF16."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    loud = torch.randperm(cols, generator=g, device="cuda")[: max(1, cols // 200)]
    x[:, loud] *= 30
    return x.to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    if case["what"].startswith("swiglu"):
        x = _activations(case["rows"], 2 * case["width"], g)
        if case["what"] == "swiglu":
            s["x"] = x
        else:   # what the forward pass kept, and the gradient that comes back
            s["codes"], s["scales"] = _mxfp8(x, case["rule"])
            s["grad"] = (torch.randn(case["rows"], case["width"], generator=g, device="cuda")
                         / 64).to(torch.bfloat16)
        return s
    s["ids"] = _choices(case, g)
    s["rows"] = _rows(case["tokens"], case["k"], case["experts"])
    if case["what"] == "route":
        return s
    s["offsets"], s["row_of"], s["entry_of"] = _route_plain(s)
    w = torch.rand(case["tokens"], case["k"], generator=g, device="cuda") + 0.05
    s["weights"] = w / w.sum(dim=1, keepdim=True) if case["weighted"] else None
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    if case["what"] != "combine":   # the tokens' rows, or the gradient of their sums
        s["x"] = _activations(case["tokens"], case["cols"], g).to(dt)
    if case["what"] != "dispatch":
        s["y"] = torch.randn(s["rows"], case["cols"], generator=g, device="cuda").to(dt)
    return s


# --------------------------------------------------------------------------- plain forms

def _route_plain(s):
    e, rows = s["experts"], s["rows"]
    flat = s["ids"].reshape(-1)
    key = torch.where(flat < 0, e, flat)
    count = torch.zeros(e + 1, dtype=torch.int64, device=flat.device)
    count.scatter_add_(0, key, torch.ones_like(key))
    padded = (count[:e] + 31) // 32 * 32
    offsets = torch.zeros(e + 1, dtype=torch.int64, device=flat.device)
    offsets[1:] = padded.cumsum(0)
    order = torch.argsort(key, stable=True)
    first = count.cumsum(0) - count          # of each expert's entries, in sorted order
    sorted_key = key[order]
    place = torch.arange(key.numel(), device=key.device) - first[sorted_key]
    row = torch.where(sorted_key < e, offsets[sorted_key] + place, -1)
    row_of = torch.empty_like(row)
    row_of[order] = row
    offsets[e] = rows                        # the last segment takes the rows left over
    entry_of = torch.full((rows + 1,), -1, dtype=torch.int64, device=key.device)
    entry_of[torch.where(row_of < 0, rows, row_of)] = torch.arange(key.numel(), device=key.device)
    return (offsets.int(), row_of.int().view(s["ids"].shape), entry_of[:rows].int())


def _dispatch_plain(s):
    """The tokens' rows in FP32, padding rows zero."""
    entry = s["entry_of"].long()
    at = entry.clamp(min=0)
    v = s["x"][at // s["k"]].float()
    if s["weights"] is not None:
        v = v * s["weights"].reshape(-1)[at][:, None]
    return v.masked_fill_((entry < 0)[:, None], 0.0)


def _two_to(e):
    """2^e in FP32 for whole e of -127 .. 127, from its bits."""
    e = e.to(torch.int32)
    return torch.where(e < -126, 1 << 22, (e + 127) << 23).to(torch.int32).view(torch.float32)


def _mxfp8(x, rule):
    """E4M3 codes and scale bytes of 1 x 32 blocks."""
    v = x.float().view(x.shape[0], -1, 32)
    amax = v.abs().amax(dim=2)
    mant, ex = torch.frexp(amax)                          # amax = mant 2^ex, 0.5 <= mant < 1
    e = ex - 9
    if rule == "ceil":                                    # the least e with amax <= 448 * 2^e
        e = e + (mant > FP8_MAX / 512).to(e.dtype)
    e = torch.where(amax > 0, e, -127).clamp(min=-127)
    q = (v * _two_to(-e)[:, :, None]).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).view(x.shape), (e + 127).to(torch.uint8)


def _tiles_of_segments(s):
    """Of each 32-row block: the rows before its segment's, its segment's 128-row tiles, and the
    tiles before its segment."""
    off = s["offsets"].long()
    tiles = (off[1:] - off[:-1] + 127) // 128
    before = tiles.cumsum(0) - tiles
    block = torch.arange(0, s["rows"], 32, device=off.device)
    e = torch.searchsorted(off[1:].contiguous(), block, right=True)
    return off[e], tiles[e], before[e]


def _swizzled(s, scales, cols, axis):
    """Scale bytes of a grouped copy in the GEMM's 128 x 4 tiles, one block of tiles a segment;
    what no segment needs is zero."""
    rows, dev = s["rows"], scales.device
    col_tiles = (cols + 127) // 128
    out = torch.zeros(((rows + 127) // 128 + s["experts"]) * col_tiles * 512,
                      dtype=torch.uint8, device=dev)
    start, tiles, before = _tiles_of_segments(s)
    if axis == "row":                                   # scales [rows, cols / 32]
        r = torch.arange(rows, device=dev)
        local = r - start.repeat_interleave(32)
        tile = before.repeat_interleave(32) + local // 128
        c = torch.arange(cols // 32, device=dev)
        at = (tile[:, None] * col_tiles + c // 4) * 512 + \
            ((local % 32) * 16 + (local % 128) // 32 * 4)[:, None] + c % 4
    else:                                               # scales [cols, rows / 32]
        block = torch.arange(0, rows, 32, device=dev)
        local = (block - start) // 32
        c = torch.arange(cols, device=dev)[:, None]
        tile = col_tiles * before + (c // 128) * tiles + local // 4
        at = tile * 512 + (c % 32) * 16 + (c % 128) // 32 * 4 + local % 4
    out[at.reshape(-1)] = scales.reshape(-1)
    return out


def _quantized(s, v):
    got = []
    if s["form"] != "col":
        q, sc = _mxfp8(v, "floor")
        got += [q, _swizzled(s, sc, s["cols"], "row")]
    if s["form"] != "row":
        q, sc = _mxfp8(v.t().contiguous(), "floor")
        got += [q, _swizzled(s, sc, s["cols"], "col")]
    return got


def _combine_plain(s):
    y, row = s["y"], s["row_of"].long()
    total = torch.zeros(s["tokens"], s["cols"], device=y.device)
    for j in range(s["k"]):
        v = y[row[:, j].clamp(min=0)].float()
        if s["weights"] is not None:
            v = v * s["weights"][:, j:j + 1]
        total += v.masked_fill_(row[:, j:j + 1] < 0, 0.0)
    return total.to(y.dtype)


def _combine_grad_plain(s):
    grad_y = _dispatch_plain(s).to(s["y"].dtype)
    row, grad_w = s["row_of"].long(), []
    x = s["x"].float()
    for j in range(s["k"]):
        dot = (x * s["y"][row[:, j].clamp(min=0)].float()).sum(dim=1)
        grad_w.append(torch.where(row[:, j] < 0, 0.0, dot))
    return grad_y, torch.stack(grad_w, dim=1)


def _swiglu_plain(s):
    g, u = s["x"].float().chunk(2, dim=1)
    h = (g * (1 / (1 + torch.exp(-g))) * u).to(torch.bfloat16)
    return (h,) + _mxfp8(s["x"], s["rule"]) if s["keep"] else (h,)


def _swiglu_grad_plain(s):
    v = s["codes"].view(torch.float8_e4m3fn).float().view(s["rows"], -1, 32)
    v = (v * _two_to(s["scales"].int() - 127)[:, :, None]).view(s["rows"], -1)
    g, u = v.chunk(2, dim=1)
    dh = s["grad"].float()
    sig = 1 / (1 + torch.exp(-g))
    silu = g * sig
    grad = torch.cat([dh * u * (sig * (1 + g * (1 - sig))), dh * silu], dim=1)
    grad = grad.to(torch.bfloat16)
    return (grad, (silu * u).to(torch.bfloat16)) if s["again"] else (grad,)


# ------------------------------------------------------------------------------ one pass

def _as_values(got):
    """E4M3 codes as what they stand for (scale bytes, flat or one for each block, stay)."""
    return [t.view(torch.float8_e4m3fn) if t.dtype == torch.uint8 and i % 2 == 0 else t
            for i, t in enumerate(got)]


def _run_plain(s):
    what = s["what"]
    if what == "route":
        return _route_plain(s)
    if what == "dispatch":
        v = _dispatch_plain(s).to(s["x"].dtype)
        return v if s["form"] == "plain" else _as_values(_quantized(s, v))
    if what == "combine":
        return _combine_plain(s)
    if what == "combine_grad":
        return _combine_grad_plain(s)
    if what == "swiglu":
        h, *kept = _swiglu_plain(s)
        return [h] + _as_values(kept)
    return _swiglu_grad_plain(s)


def _run_own(s):
    import mxfp8_block_scaled_05_gb300 as m
    what = s["what"]
    if what == "route":
        return tuple(m.route(s["ids"], s["experts"]))
    if what == "swiglu":
        rule = m.RULE_CEIL if s["rule"] == "ceil" else m.RULE_FLOOR
        h, *kept = m.swiglu(s["x"], checkpoint=s["keep"], rule=rule)
        return [h] + (_as_values(kept) if s["keep"] else [])
    if what == "swiglu_grad":
        grad, h = m.swiglu_backward(s["grad"], s["codes"], s["scales"], recompute=s["again"])
        return (grad, h) if s["again"] else (grad,)
    plan = m.RoutePlan(s["offsets"], s["row_of"], s["entry_of"])
    if what == "combine":
        return m.combine(s["y"], plan, s["weights"])
    if what == "combine_grad":
        return m.combine_backward(s["x"], s["y"], plan, s["weights"])
    if s["form"] == "plain":
        return m.dispatch(s["x"], plan, s["weights"])
    if s["form"] == "dual":
        return _as_values(m.quantize_dispatch_dual(s["x"], plan, s["weights"]))
    axis = m.ROW if s["form"] == "row" else m.COL
    return _as_values(m.quantize_dispatch(s["x"], plan, axis, s["weights"]))


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------------ work and 64 bits

def work(case):
    what = case["what"]
    if what.startswith("swiglu"):
        n = float(case["rows"] * case["width"])
        kept = 2 * n * 33 / 32
        if what == "swiglu":
            return dict(bytes=6 * n + (kept if case["keep"] else 0), flops=6 * n)
        return dict(bytes=6 * n + kept + (2 * n if case["again"] else 0), flops=12 * n)
    entries = float(case["tokens"] * case["k"])
    rows = _rows(case["tokens"], case["k"], case["experts"])
    if what == "route":
        return dict(bytes=12 * entries + 4 * rows + 4 * case["experts"], flops=2 * entries)
    c, size = case["cols"], 2 if case["dtype"] == "bf16" else 4
    live = entries * (1 - case["dropped"])
    if what == "dispatch":
        written = {"plain": size, "row": 33 / 32, "col": 33 / 32, "dual": 33 / 16}[case["form"]]
        return dict(bytes=case["tokens"] * c * size + rows * (c * written + 4) + 4 * entries,
                    flops=live * c)
    if what == "combine":
        return dict(bytes=(live + case["tokens"]) * c * size + 8 * entries, flops=2 * live * c)
    return dict(bytes=(live + case["tokens"] + rows) * c * size + 12 * entries + 4 * rows,
                flops=3 * live * c)


def _power(e):
    """2^e in 64 bits for whole e, from its bits."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_grid(v):
    """v rounded to the nearest E4M3 value, ties to even, in 64 bits."""
    a = v.abs().clamp(max=FP8_MAX)
    _, ex = torch.frexp(a)
    step = _power((ex - 1).clamp(min=-6) - 3)
    return torch.copysign((a / step).round() * step, v)   # round() takes ties to even


def _exact_codes(v, rule):
    """E4M3 values of 1 x 32 blocks of BF16 values given in 64 bits."""
    b = v.reshape(v.shape[0], -1, 32)
    peak = b.abs().amax(dim=2, keepdim=True)
    _, ex = torch.frexp(peak)
    e = ex.to(torch.int64) - 9                  # 2^(e + 8) <= peak < 2^(e + 9)
    if rule == "ceil":                          # nothing above 448 of the block's scale
        e = torch.where(peak > FP8_MAX * _power(e), e + 1, e)
    e = torch.where(peak > 0, e, -127).clamp(min=-127)
    return _exact_grid(b / _power(e)).reshape(v.shape)


def exact(case, seed):
    s = prepare(case, seed)
    what = s["what"]
    if what == "route":
        return None
    if what == "swiglu":
        x = s["x"].double()
        f = s["width"]
        h = torch.sigmoid(x[:, :f]) * x[:, :f] * x[:, f:]
        return [h, _exact_codes(x, s["rule"]), None] if s["keep"] else [h]
    if what == "swiglu_grad":
        scale = _power(s["scales"].to(torch.int64) - 127).repeat_interleave(32, 1)
        x = s["codes"].view(torch.float8_e4m3fn).double() * scale
        del scale
        f = s["width"]
        g, u, dh = x[:, :f], x[:, f:], s["grad"].double()
        sig = torch.sigmoid(g)
        out = torch.empty_like(x)
        out[:, :f] = dh * u * (sig + g * sig * torch.sigmoid(-g))
        out[:, f:] = dh * g * sig
        return (out, g * sig * u) if s["again"] else (out,)
    k, rows = s["k"], s["rows"]
    w = s["weights"].double() if s["weights"] is not None else \
        torch.ones(s["tokens"], k, dtype=torch.float64, device="cuda")
    row = s["row_of"].long()
    live = row >= 0
    if what == "combine":
        total = torch.zeros(s["tokens"], s["cols"], dtype=torch.float64, device="cuda")
        for j in range(k):
            t = live[:, j].nonzero()[:, 0]
            total[t] += w[t, j:j + 1] * s["y"][row[t, j]].double()
        return total
    spread = torch.zeros(rows, s["cols"], dtype=torch.float64, device="cuda")
    x = s["x"].double()
    for j in range(k):
        t = live[:, j].nonzero()[:, 0]
        spread[row[t, j]] = x[t] * w[t, j:j + 1]
    if what == "dispatch":
        if s["form"] == "plain":
            return spread
        if s["weights"] is not None:   # the rows are BF16 before they are put on the grid
            return None
        got = []
        if s["form"] != "col":
            got += [_exact_codes(spread, "floor"), None]
        if s["form"] != "row":
            got += [_exact_codes(spread.t(), "floor"), None]
        return got
    grad_w = torch.zeros(s["tokens"], k, dtype=torch.float64, device="cuda")
    for j in range(k):
        t = live[:, j].nonzero()[:, 0]
        grad_w[t, j] = (x[t] * s["y"][row[t, j]].double()).sum(dim=1)
    return spread, grad_w
