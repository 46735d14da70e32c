"""Cases and plain forms of the block-scaled FP8 product and of the token log probabilities.

Four operators, as the package offers them:

- ``blockwise_gemm``: C = deq(A) deq(B)^T on E4M3 codes whose scales cover 128 values along
  the reduction (A: 1 x 128 blocks; B: 128 x 128 blocks, or 1 x 128 for a weight gradient).
- ``quantize_blockwise_1d`` (``_dual``) and ``quantize_blockwise_dual``: the quantizers that
  write those operands from BF16, row-wise, transposed, or both from one read.
- ``token_logprobs``: log probability of a given token, entropy and the likeliest
  alternatives of each row of logits.
- ``token_logprobs_backward``: the gradient of those with respect to the logits.

``own`` chooses between the plain form (elementary torch operations in 32 bits) and the
package's kernels. Sizes are the linear layers that the package's workloads name, and
generic vocabularies.
"""
import math

import torch

own = False

# Linear layers of the package's workloads as (N = out_features, K = in_features).
QKV, O_PROJ, GATE_UP, DOWN = (6144, 4096), (4096, 4096), (24576, 4096), (4096, 12288)
FP8_MAX = 448.0
MOST_FLOPS = 2.0 * 4096 * GATE_UP[0] * GATE_UP[1]   # the largest listed product
MOST_LOGIT_BYTES = 4096 * 131072 * 2                # the largest listed logits


# ------------------------------------------------------------------------------- cases

def listed():
    return [
        # one token through an attention output projection while a sampler decodes
        dict(name="gemm_decode_1", what="gemm", op="fprop", m=1, n=O_PROJ[0], k=O_PROJ[1],
             out="bf16", scale="fp32"),
        # a small, ragged decode batch through the widest projection
        dict(name="gemm_decode_37", what="gemm", op="fprop", m=37, n=GATE_UP[0], k=GATE_UP[1],
             out="bf16", scale="fp32"),
        # the data gradient of a down projection for an odd number of packed tokens
        dict(name="gemm_dgrad_1021", what="gemm", op="dgrad", m=1021, n=DOWN[1], k=DOWN[0],
             out="bf16", scale="pow2"),
        # the forward product of a full micro-batch through the widest projection
        dict(name="gemm_fprop_4096", what="gemm", op="fprop", m=4096, n=GATE_UP[0],
             k=GATE_UP[1], out="bf16", scale="pow2"),
        # the weight gradient of a projection over an odd number of tokens, kept in FP32
        dict(name="gemm_wgrad_4001", what="gemm", op="wgrad", m=QKV[0], n=QKV[1], k=4001,
             out="fp32", scale="pow2"),
        # a decode batch's activations on their way into a product
        dict(name="quant_row_37", what="quant", form="row", rows=37, cols=4096, scale="fp32"),
        # a micro-batch's activations, both copies, on the way into forward and weight gradient
        dict(name="quant_dual_4096", what="quant", form="dual", rows=4096, cols=12288,
             scale="pow2"),
        # one sampled token: its log probability and the usual number of reported alternatives
        dict(name="logprob_1", what="logprob", rows=1, vocab=131072, ld=131072, dtype="bf16",
             top=20, temperature=0.7, masked=0.0),
        # constrained sampling: FP32 logits, most of an odd vocabulary masked, one row empty
        dict(name="logprob_masked_253", what="logprob", rows=253, vocab=50021, ld=50021,
             dtype="fp32", top=5, temperature=1.0, masked=0.6),
        # scoring a micro-batch of sampled tokens under the learner
        dict(name="logprob_4096", what="logprob", rows=4096, vocab=131072, ld=131072,
             dtype="bf16", top=8, temperature=1.0, masked=0.0),
        # the policy gradient of a few sequences, an odd vocabulary inside padded rows
        dict(name="logprob_grad_509", what="grad", rows=509, vocab=32003, ld=32064,
             dtype="fp32", top=4, temperature=0.8, masked=0.0),
        # the policy gradient of a micro-batch
        dict(name="logprob_grad_4096", what="grad", rows=4096, vocab=131072, ld=131072,
             dtype="bf16", top=0, temperature=1.0, masked=0.0),
    ]


def _size(rng, lo, hi, unit=1):
    """A multiple of `unit` between `unit * lo` and `unit * hi`, spread over its logarithm.
    No multiple of three: those of the listed layers stay apart from the drawn ones."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    n = min(hi, max(lo, n))
    return unit * (n if n % 3 else n - 1)


def draw(rng):
    what = rng.choice(["gemm", "gemm", "quant", "logprob", "grad"])
    scale = rng.choice(["fp32", "pow2"])
    if what == "gemm":
        op = rng.choice(["fprop", "dgrad", "wgrad"])
        while True:
            n, k, m = _size(rng, 8, 3000, 8), _size(rng, 8, 760, 16), _size(rng, 1, 8192)
            if op == "wgrad":   # features x features, reduced over the tokens
                m, k = _size(rng, 8, 1500, 8), m
            if 2.0 * m * n * k <= MOST_FLOPS:
                break
        return dict(what=what, op=op, m=m, n=n, k=k, out=rng.choice(["bf16", "fp32"]),
                    scale=scale)
    if what == "quant":
        form = rng.choice(["row", "col", "dual", "weight_dual"])
        rows = _size(rng, 1, 512, 16) if form == "weight_dual" else _size(rng, 1, 8192)
        return dict(what=what, form=form, rows=rows, cols=_size(rng, 8, 760, 16), scale=scale)
    dtype = rng.choice(["bf16", "fp32"])
    while True:
        rows, vocab = _size(rng, 1, 4096), _size(rng, 1000, 160000)
        # packed rows, or longer ones that start on 64-byte boundaries
        ld = vocab if rng.random() < 0.5 else 32 * (vocab // 32 + (1 if vocab // 32 % 3 < 2 else 2))
        if rows * ld * (2 if dtype == "bf16" else 4) <= MOST_LOGIT_BYTES:
            break
    return dict(what=what, rows=rows, vocab=vocab, ld=ld, dtype=dtype,
                top=rng.choice([0, 1, 5, 20, 32]), temperature=rng.choice([0.6, 1.0, 1.3]),
                masked=rng.choice([0.0, 0.0, 0.5]))


def _pad16(n):
    return (n + 15) // 16 * 16


# ------------------------------------------------------------------- quantizers, plainly

def _pow2_inverse(amax):
    """2^ceil(log2(amax / 448)), at least 2^-127; 1 for zero."""
    mant, ex = torch.frexp(amax)                  # amax = mant * 2^ex, 0.5 <= mant < 1
    e = ex - 9 + (mant > FP8_MAX / 512).to(ex.dtype)
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e.clamp(min=-127)),
                       torch.ones_like(amax))


def _scale_pair(amax, scale):
    """The factor a block is multiplied with, and its inverse."""
    if scale == "pow2":
        inv = _pow2_inverse(amax)
        return 1 / inv, inv
    s = torch.where(amax > 0, (FP8_MAX / amax).clamp(max=torch.finfo(torch.float32).max),
                    torch.ones_like(amax))
    return s, 1 / s


def _blocks(x, br, bc):
    """[rows, cols] -> [row blocks, br, column blocks, bc], zero-padded."""
    r, c = x.shape
    x = torch.nn.functional.pad(x, (0, -c % bc, 0, -r % br))
    return x.view(x.shape[0] // br, br, x.shape[1] // bc, bc)


def _quantize(x, br, bc, scale):
    """E4M3 codes [rows, cols] and scale inverses [row blocks, column blocks]."""
    b = _blocks(x.float(), br, bc)
    s, inv = _scale_pair(b.abs().amax(dim=(1, 3)), scale)
    q = (b * s[:, None, :, None]).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
    q = q.view(torch.uint8).view(b.shape[0] * br, b.shape[2] * bc)
    return q[: x.shape[0], : x.shape[1]].contiguous(), inv


def _quantize_1d(x, axis, scale):
    """As quantize_blockwise_1d: codes with the blocked dimension last (a transposed copy is
    padded with zeros to a multiple of 16), scale inverses [blocks, rows of the codes]."""
    if axis == "row":
        q, inv = _quantize(x, 1, 128, scale)
        return q, inv.t().contiguous()
    q, inv = _quantize(x, 128, 1, scale)
    return torch.nn.functional.pad(q, (0, 0, 0, -x.shape[0] % 16)).t().contiguous(), inv


def _deq_1d(q, inv):
    v = q.view(torch.float8_e4m3fn).float()
    return v * inv.t().repeat_interleave(128, 1)[:, : v.shape[1]]


def _deq_2d(q, inv):
    v = q.view(torch.float8_e4m3fn).float()
    return v * inv.repeat_interleave(128, 0).repeat_interleave(128, 1)[: v.shape[0], : v.shape[1]]


# ----------------------------------------------------------------------- inputs of a case

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _activations(rows, cols, g):
    """N(0, 1) with a few outlier features, in BF16."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    loud = torch.randperm(cols, generator=g, device="cuda")[: max(1, cols // 200)]
    x[:, loud] *= 30
    return x.to(torch.bfloat16)


def _logits(case, g):
    rows, vocab, ld = case["rows"], case["vocab"], case["ld"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    buf = torch.empty(rows, ld, dtype=dt, device="cuda")
    for r0 in range(0, rows, 512):
        x = torch.randn(min(512, rows - r0), ld, generator=g, device="cuda")
        buf[r0:r0 + 512] = (x * 2.5).to(dt)
    x = buf[:, :vocab]
    likely = torch.randint(vocab, (rows, 4), generator=g, device="cuda")
    x.scatter_add_(1, likely, torch.full((rows, 4), 8.0, dtype=dt, device="cuda"))
    if case["masked"]:
        for r0 in range(0, rows, 512):
            part = x[r0:r0 + 512]
            gone = torch.rand(part.shape, generator=g, device="cuda") < case["masked"]
            part.masked_fill_(gone, -math.inf)
        if rows > 1:
            x[rows // 2] = -math.inf
    # what was sampled: a likely token, or any; one in eight is part of a prompt, not scored
    target = torch.where(torch.rand(rows, generator=g, device="cuda") < 0.7, likely[:, 0],
                         torch.randint(vocab, (rows,), generator=g, device="cuda"))
    if rows > 1:
        target[torch.rand(rows, generator=g, device="cuda") < 0.125] = -1
    return x, target


def prepare(case, seed):
    g = _generator(seed)
    what = case["what"]
    s = dict(case)
    if what == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        if case["op"] == "wgrad":
            dy = torch.randn(k, m, generator=g, device="cuda").to(torch.bfloat16)
            s["a"], s["sa"] = _quantize_1d(dy, "col", case["scale"])
            s["b"], s["sb"] = _quantize_1d(_activations(k, n, g), "col", case["scale"])
        else:
            s["a"], s["sa"] = _quantize_1d(_activations(m, k, g), "row", case["scale"])
            w = (torch.randn(n, k, generator=g, device="cuda") * 0.02).to(torch.bfloat16)
            s["b"], s["sb"] = _quantize(w, 128, 128, case["scale"])
    elif what == "quant":
        if case["form"] == "weight_dual":
            x = torch.randn(case["rows"], case["cols"], generator=g, device="cuda") * 0.02
            s["x"] = x.to(torch.bfloat16)
        else:
            s["x"] = _activations(case["rows"], case["cols"], g)
    else:
        s["x"], s["target"] = _logits(case, g)
        if what == "grad":
            rows, top = case["rows"], case["top"]
            rand = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
            s["g_logprob"] = rand(rows) / 8
            s["g_entropy"] = rand(rows) * 0.01
            # what the forward call left behind
            fwd = _logprob_plain(s["x"], s["target"], case["temperature"], top)
            s["entropy"], s["stats"] = fwd["entropy"], fwd["stats"]
            s["top_id"] = fwd["top_id"] if top else None
            s["g_top"] = rand(rows, top) / 8 if top else None
    return s


# --------------------------------------------------------------- log probabilities, plainly

def _top(x, k):
    """Places of the k largest values of each row, ties to the lowest place; -1 where fewer
    than k are above -inf."""
    bits = (x + 0.0).view(torch.int32).to(torch.int64)
    order = torch.where(bits >= 0, bits, -(bits & 0x7FFFFFFF))
    vocab = x.shape[1]
    key = order * (1 << 20) + (vocab - 1 - torch.arange(vocab, device=x.device))
    if vocab < k:
        key = torch.nn.functional.pad(key, (0, k - vocab), value=-(1 << 62))
    best = key.topk(k, dim=1).values
    place = vocab - 1 - (best & ((1 << 20) - 1))
    value = x.gather(1, place.clamp(0, vocab - 1))
    none = (value == -math.inf) | (best == -(1 << 62))
    return torch.where(none, -1, place)


def _logprob_plain(x, target, temperature, top):
    x = x.float()
    peak = x.amax(dim=1, keepdim=True)
    empty = peak == -math.inf
    d = (x - torch.where(empty, 0.0, peak)) * (1.0 / temperature)
    e = d.exp()
    total = e.sum(dim=1, keepdim=True)
    log_total = torch.where(empty, 0.0, total.log())
    weighted = (e * torch.where(e > 0, d, 0.0)).sum(dim=1, keepdim=True)
    entropy = torch.where(empty, 0.0, log_total - weighted / total)
    chosen = d.gather(1, target.clamp(min=0)[:, None]) - log_total
    logprob = torch.where(target[:, None] < 0, 0.0, chosen)
    got = dict(logprob=logprob[:, 0], entropy=entropy[:, 0],
               stats=torch.cat([peak, log_total], dim=1))
    if top:
        place = _top(x, top)
        value = d.gather(1, place.clamp(min=0)) - log_total
        got["top_logprob"] = torch.where(place < 0, -math.inf, value)
        got["top_id"] = place
    return got


def _grad_plain(s):
    inv_t = 1.0 / s["temperature"]
    x = s["x"].float()
    peak = x.amax(dim=1, keepdim=True)
    empty = peak == -math.inf
    d = (x - torch.where(empty, 0.0, peak)) * inv_t
    e = d.exp()
    total = torch.where(empty, 1.0, e.sum(dim=1, keepdim=True))
    p = e / total
    logp = torch.where(p > 0, d - total.log(), 0.0)
    entropy = -(p * logp).sum(dim=1, keepdim=True)
    g = torch.where((s["target"] < 0)[:, None] | empty, 0.0, s["g_logprob"][:, None])
    h = s["g_entropy"][:, None]
    mass = g
    if s["top"]:
        listed_top = s["top_id"] >= 0
        g_top = torch.where(listed_top, s["g_top"], 0.0)
        mass = mass + g_top.sum(dim=1, keepdim=True)
    z = -p * (mass + h * (logp + entropy))
    z.scatter_add_(1, s["target"].clamp(min=0)[:, None], g)
    if s["top"]:
        z.scatter_add_(1, s["top_id"].clamp(min=0), g_top)
    return (z * inv_t).to(s["x"].dtype)


# ------------------------------------------------------------------------------ one pass

def _run_plain(s):
    if s["what"] == "gemm":
        a = _deq_1d(s["a"], s["sa"])
        b = _deq_1d(s["b"], s["sb"]) if s["op"] == "wgrad" else _deq_2d(s["b"], s["sb"])
        c = a @ b.t()
        return c.to(torch.bfloat16) if s["out"] == "bf16" else c
    if s["what"] == "quant":
        x, scale = s["x"], s["scale"]
        if s["form"] == "weight_dual":
            q, inv = _quantize(x, 128, 128, scale)
            got = [q, inv, q.t().contiguous(), inv.t().contiguous()]
        else:
            got = []
            if s["form"] != "col":
                got += _quantize_1d(x, "row", scale)
            if s["form"] != "row":
                got += _quantize_1d(x, "col", scale)
        return [t.view(torch.float8_e4m3fn) if t.dtype == torch.uint8 else t for t in got]
    if s["what"] == "logprob":
        return _logprob_plain(s["x"], s["target"], s["temperature"], s["top"])
    return _grad_plain(s)


def _run_own(s):
    import mxfp8_block_scaled_05_gb300 as m
    if s["what"] == "gemm":
        op = {"fprop": m.FPROP, "dgrad": m.DGRAD, "wgrad": m.WGRAD}[s["op"]]
        return m.blockwise_gemm(s["a"], s["sa"], s["b"], s["sb"], op,
                                m.OUT_BF16 if s["out"] == "bf16" else m.OUT_FP32)
    if s["what"] == "quant":
        scale = m.BW_POW2 if s["scale"] == "pow2" else m.BW_FP32
        if s["form"] == "dual":
            got = m.quantize_blockwise_1d_dual(s["x"], scale)
        elif s["form"] == "weight_dual":
            got = m.quantize_blockwise_dual(s["x"], scale)
        else:
            got = m.quantize_blockwise_1d(s["x"], m.ROW if s["form"] == "row" else m.COL, scale)
        return [t.view(torch.float8_e4m3fn) if t.dtype == torch.uint8 else t for t in got]
    if s["what"] == "logprob":
        r = m.token_logprobs(s["x"], s["target"], temperature=s["temperature"], top=s["top"])
        got = dict(logprob=r.logprob, entropy=r.entropy, stats=r.stats)
        if s["top"]:
            got.update(top_logprob=r.top_logprob, top_id=r.top_id)
        return got
    return m.token_logprobs_backward(s["x"], s["target"], s["stats"], s["entropy"],
                                     s["g_logprob"], grad_entropy=s["g_entropy"],
                                     top_id=s["top_id"], grad_top=s["g_top"],
                                     temperature=s["temperature"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------------ work and 64 bits

def work(case):
    if case["what"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        kb = -(-k // 128)
        scales = m * kb + (n * kb if case["op"] == "wgrad" else -(-n // 128) * kb)
        return dict(bytes=(m + n) * k + 4 * scales + m * n * (2 if case["out"] == "bf16" else 4),
                    flops=2.0 * m * n * k)
    if case["what"] == "quant":
        r, c, form = case["rows"], case["cols"], case["form"]
        rb, cb = -(-r // 128), -(-c // 128)
        n = r * c
        if form == "weight_dual":
            return dict(bytes=4 * n + 8 * rb * cb, flops=3.0 * n)
        total = 2 * n
        total += (n + 4 * cb * r) if form != "col" else 0
        total += (n + 4 * rb * c) if form != "row" else 0
        return dict(bytes=total, flops=(4.0 if form == "dual" else 2.0) * n)
    n = case["rows"] * case["vocab"]
    size = 2 if case["dtype"] == "bf16" else 4
    if case["what"] == "logprob":
        return dict(bytes=n * size + case["rows"] * (8 + 16 + 12 * case["top"]), flops=6.0 * n)
    return dict(bytes=2 * n * size + case["rows"] * (28 + 12 * case["top"]), flops=8.0 * n)


def _exact_grid(v):
    """v rounded to the nearest E4M3 value, ties to even, in 64 bits."""
    a = v.abs().clamp(max=FP8_MAX)
    _, ex = torch.frexp(a)
    step = torch.ldexp(torch.ones_like(a), (ex - 1).clamp(min=-6) - 3)
    return torch.copysign((a / step).round() * step, v)   # round() takes ties to even


def _exact_quant(x, br, bc, scale):
    b = _blocks(x.double(), br, bc)
    amax = b.abs().amax(dim=(1, 3))
    inv = torch.where(amax > 0, amax / FP8_MAX, torch.ones_like(amax))
    if scale == "pow2":
        mant, ex = torch.frexp(inv)
        inv = torch.ldexp(torch.ones_like(inv), torch.where(mant > 0.5, ex, ex - 1))
    q = _exact_grid(b / inv[:, None, :, None]).view(b.shape[0] * br, b.shape[2] * bc)
    return q[: x.shape[0], : x.shape[1]].contiguous(), inv


def exact(case, seed):
    s = prepare(case, seed)
    if s["what"] == "gemm":
        def rows_of(q, inv):
            v = q.view(torch.float8_e4m3fn).double()
            for kb in range(inv.shape[0]):
                v[:, 128 * kb:128 * kb + 128] *= inv[kb].double()[:, None]
            return v
        a = rows_of(s["a"], s["sa"])
        sb = s["sb"] if s["op"] == "wgrad" else \
            s["sb"].t().repeat_interleave(128, 1)[:, : s["b"].shape[0]]
        return a @ rows_of(s["b"], sb).t()
    if s["what"] == "quant":
        x, scale = s["x"], s["scale"]
        if s["form"] == "weight_dual":
            q, inv = _exact_quant(x, 128, 128, scale)
            return [q, inv, q.t(), inv.t()]
        got = []
        if s["form"] != "col":
            q, inv = _exact_quant(x, 1, 128, scale)
            got += [q, inv.t()]
        if s["form"] != "row":
            q, inv = _exact_quant(x, 128, 1, scale)
            got += [torch.nn.functional.pad(q, (0, 0, 0, -x.shape[0] % 16)).t(), inv]
        return got
    # log probabilities and their gradient, some rows at a time
    t, parts = float(s["temperature"]), []
    for r0 in range(0, case["rows"], 256):
        at = slice(r0, r0 + 256)
        x, target = s["x"][at].double(), s["target"][at]
        peak = x.max(dim=1).values
        empty = peak.isinf()
        z = x / t
        lse = torch.logsumexp(z, dim=1)
        logp = torch.where(empty[:, None], -math.inf, z - lse[:, None])
        p = logp.exp()
        logp0 = torch.where(p > 0, logp, 0.0)
        entropy = -(p * logp0).sum(dim=1)
        if s["what"] == "logprob":
            chosen = logp.gather(1, target.clamp(min=0)[:, None])[:, 0]
            got = dict(logprob=torch.where(target < 0, 0.0, chosen), entropy=entropy,
                       stats=torch.stack([peak, torch.where(empty, 0.0, lse - peak / t)], dim=1))
            if s["top"]:
                got["top_logprob"] = logp.topk(s["top"], dim=1).values
            parts.append(got)
            continue
        g = torch.where((target < 0) | empty, 0.0, s["g_logprob"][at].double())
        dz = -p * (g[:, None] + s["g_entropy"][at].double()[:, None] * (logp0 + entropy[:, None]))
        dz.scatter_add_(1, target.clamp(min=0)[:, None], g[:, None])
        if s["top"]:
            ids = s["top_id"][at]
            gt = torch.where(ids < 0, 0.0, s["g_top"][at].double())
            dz -= p * gt.sum(dim=1, keepdim=True)
            dz.scatter_add_(1, ids.clamp(min=0), gt)
        parts.append(dz / t)
    if s["what"] == "grad":
        return torch.cat(parts)
    got = {key: torch.cat([q[key] for q in parts]) for key in parts[0]}
    if s["top"]:
        got["top_id"] = None
    return got
