"""Measured cases of routing by scores with its gradient, and of products with 4-bit integer weights.

Four groups of calls, each with a plain form in elementary torch operations
(`own` false) and the calls that a user makes of the library (`own` true):
the choice of experts from router logits (softmax or sigmoid scores, a bias,
groups, top-k, weights), its gradient, the quantisation of weights to 4-bit
codes with group scales (with the dequantisation that reads them back), and the
grouped product of bf16 rows with such weights.
"""
import math

import torch

own = False


# ------------------------------------------------------------------ cases
def listed():
    return [
        # routing of a decode batch, as bias-balanced routers with groups do it: latency counts
        dict(name="select, decode", op="select", T=128, E=256, k=8, score="sigmoid", bias=True, groups=8, group_k=4,
             group_top=2, renorm=True, dtype="f32", scores=False, masked=False),
        # routing of a prefill chunk by softmax and top-k alone
        dict(name="select, prefill", op="select", T=16384, E=256, k=8, score="softmax", bias=False, groups=1, group_k=1,
             group_top=1, renorm=True, dtype="bf16", scores=False, masked=False),
        # a training batch: padded rows and experts left out, scores kept for a balance loss
        dict(name="select, training", op="select", T=131072, E=160, k=6, score="sigmoid", bias=True, groups=8, group_k=3,
             group_top=2, renorm=True, dtype="f32", scores=True, masked=True),
        # gradient of a small step
        dict(name="select gradient, small", op="select_bwd", T=500, E=64, k=6, score="softmax", renorm=False,
             dtype="f32", dl="f32", dscores=False, masked=False),
        # gradient of a training batch, with the gradient of a balance loss
        dict(name="select gradient, training", op="select_bwd", T=131072, E=256, k=8, score="sigmoid", renorm=True,
             dtype="bf16", dl="bf16", dscores=True, masked=True),
        # one projection of one expert converted by rows, with zero points
        dict(name="w4 quantise, rows", op="quant", B=1, R=1536, C=5120, trans=False, group=128, zeros=True, dtype="bf16",
             sdtype="bf16"),
        # a set of expert weights converted once, from [K, N] to K-contiguous codes
        dict(name="w4 quantise, weights", op="quant", B=32, R=5120, C=1536, trans=True, group=64, zeros=False,
             dtype="bf16", sdtype="bf16"),
        # one decoded token through one projection of its 8 experts: bound by the code stream
        dict(name="w4 product, one token", op="product", T=1, k=8, E=256, K=5120, N=1536, group=128, zeros=False,
             gather=True, out="bf16", sdtype="bf16"),
        # one token through a dense projection (one expert), with zero points
        dict(name="w4 product, dense vector", op="product", T=1, k=1, E=1, K=5120, N=16384, group=64, zeros=True,
             gather=False, out="bf16", sdtype="bf16"),
        # a decode batch: about 100 experts with one or two rows each
        dict(name="w4 product, decode", op="product", T=16, k=8, E=256, K=5120, N=1536, group=128, zeros=True,
             gather=True, out="bf16", sdtype="bf16"),
        # a middling batch over widths that are not multiples of a tile, fp32 results for the weighted sum
        dict(name="w4 product, ragged", op="product", T=333, k=6, E=48, K=1440, N=2056, group=32, zeros=True,
             gather=True, out="f32", sdtype="f32"),
        # a prefill chunk: bound by the matrix instructions
        dict(name="w4 product, prefill", op="product", T=4096, k=8, E=64, K=5120, N=2560, group=128, zeros=False,
             gather=True, out="bf16", sdtype="bf16"),
    ]


def draw(rng):
    def size(lo, hi, unit):
        return max(unit, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / unit)) * unit)

    op = rng.choice(["select", "select", "select_bwd", "quant", "product", "product", "product"])
    while True:
        if op in ("select", "select_bwd"):
            groups = rng.choice([1, 1, 4, 8, 10])
            E = size(8, 256 // groups if op == "select" and groups > 1 else 256, 1)
            if op == "select":
                E = E * groups if groups > 1 else E
                group_k = rng.randint(max(1, -(-groups // 3)), groups)
                k = rng.randint(1, min(8, group_k * (E // groups)))
                c = dict(op=op, T=size(1, 131072, 1), E=E, k=k, score=rng.choice(["softmax", "sigmoid"]),
                         bias=rng.random() < 0.5, groups=groups, group_k=group_k, group_top=rng.randint(1, 2),
                         renorm=rng.random() < 0.7, dtype=rng.choice(["f32", "bf16"]), scores=rng.random() < 0.3,
                         masked=rng.random() < 0.4)
            else:
                c = dict(op=op, T=size(1, 131072, 1), E=E, k=rng.randint(1, min(8, E)),
                         score=rng.choice(["softmax", "sigmoid"]), renorm=rng.random() < 0.7,
                         dtype=rng.choice(["f32", "bf16"]), dl=rng.choice(["f32", "bf16"]),
                         dscores=rng.random() < 0.4, masked=rng.random() < 0.4)
            top = dict(bytes=2.9e8, flops=1e12)
        elif op == "quant":
            trans, group = rng.random() < 0.5, rng.choice([32, 64, 128])
            a, b = size(128, 5120, group), size(8, 2560, 8)
            c = dict(op=op, B=size(1, 32, 1) if trans else 1, R=a if trans else size(1, 16384, 1), C=b if trans else a,
                     trans=trans, group=group, zeros=rng.random() < 0.5, dtype=rng.choice(["bf16", "bf16", "f32"]),
                     sdtype=rng.choice(["bf16", "bf16", "f32"]))
            top = dict(bytes=1.1e9, flops=1e12)
        else:
            E, group = size(1, 256, 1), rng.choice([32, 64, 128])
            c = dict(op=op, T=size(1, 4096, 1), k=rng.randint(1, min(8, E)), E=E, K=size(128, 5120, group),
                     N=size(64, 2560, 8), group=group, zeros=rng.random() < 0.5, gather=rng.random() < 0.7,
                     out=rng.choice(["bf16", "bf16", "f32"]), sdtype=rng.choice(["bf16", "bf16", "f32"]))
            top = dict(bytes=1.2e9, flops=8.6e11)
        w = work(c)
        if w["bytes"] <= top["bytes"] and w["flops"] <= top["flops"]:
            return c


def _touched(c):
    """Experts that have rows, as uniform routing gives them on average."""
    return c["E"] * (1 - (1 - c["k"] / c["E"]) ** c["T"])


def work(c):
    op, size = c["op"], {"bf16": 2, "f32": 4}
    if op == "select":
        n, P = c["T"] * c["E"], c["T"] * c["k"]
        return dict(bytes=n * (size[c["dtype"]] + (4 if c["scores"] else 0)) + 8 * P, flops=12.0 * n)
    if op == "select_bwd":
        n, P = c["T"] * c["E"], c["T"] * c["k"]
        return dict(bytes=n * (size[c["dtype"]] + size[c["dl"]] + (4 if c["dscores"] else 0)) + 8 * P, flops=12.0 * n)
    per = 0.5 + (size[c["sdtype"]] + (1 if c["zeros"] else 0)) / c["group"]
    if op == "product":
        P = c["T"] * c["k"]
        rows = c["T"] if c["gather"] else P
        return dict(bytes=rows * c["K"] * 2 + _touched(c) * c["K"] * c["N"] * per + P * c["N"] * size[c["out"]],
                    flops=2.0 * P * c["K"] * c["N"])
    n = c["B"] * c["R"] * c["C"]
    return dict(bytes=n * (2 * size[c["dtype"]] + per), flops=4.0 * n)


# ------------------------------------------------------------------ inputs
_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_INF = float("inf")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c, op = dict(case), case["op"]

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device="cuda", dtype=dtype) * scale).to(dtype)

    if op in ("select", "select_bwd"):
        T, E, k = c["T"], c["E"], c["k"]
        # favoured experts and tokens of different sharpness
        logits = (normal(T, E) + 0.5 * normal(E)) * (0.5 + 2 * torch.rand(T, 1, generator=g, device="cuda"))
        if c["masked"]:  # padded rows at the end, and experts that some tokens may not take
            logits[torch.rand(T, E, generator=g, device="cuda") < 0.05] = -_INF
            logits[T - T // 16:] = -_INF
        s = dict(c=c, logits=logits.to(_DTYPES[c["dtype"]]))
        if op == "select":
            s["bias"] = normal(E, scale=0.1) if c["bias"] else None
            return s
        picked = torch.where(s["logits"] == -_INF, -1.0, torch.rand(T, E, generator=g, device="cuda"))
        top = torch.sort(picked, dim=1, descending=True)
        s["ids"] = torch.where(top.values >= 0, top.indices, -1)[:, :k].to(torch.int32).contiguous()
        s["dw"] = normal(T, k, scale=0.1)
        s["dscores"] = normal(T, E, scale=0.01) if c["dscores"] else None
        return s
    if op == "quant":
        x = normal(c["B"], c["R"], c["C"], scale=0.7, dtype=_DTYPES[c["dtype"]])
        # outlier columns, as weights have them: the groups' scales differ widely
        x *= torch.exp2(torch.randint(-3, 4, (c["C"],), generator=g, device="cuda").to(x.dtype))
        return dict(c=c, x=x if c["trans"] else x[0])
    T, k, E, K, N = c["T"], c["k"], c["E"], c["K"], c["N"]
    # experts of each token (a mildly uneven load), and the rows sorted by expert
    ids = (torch.randn(T, E, generator=g, device="cuda") + 0.4 * torch.randn(E, generator=g, device="cuda"))
    ids = ids.topk(k, dim=1).indices.reshape(-1)
    order = torch.sort(ids, stable=True).indices
    counts = torch.zeros(E, dtype=torch.int64, device="cuda").index_add_(0, ids, torch.ones_like(ids))
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    s = dict(c=c, offsets=offsets, widest=int(counts.max()), index=order.to(torch.int32) if c["gather"] else None)
    s["a"] = normal(T if c["gather"] else T * k, K, dtype=torch.bfloat16)
    s["codes"] = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda")
    s["scales"] = torch.empty(E, N, K // c["group"], dtype=_DTYPES[c["sdtype"]], device="cuda")
    s["zeros"] = torch.empty(E, N, K // c["group"], dtype=torch.uint8, device="cuda") if c["zeros"] else None
    for e in range(E):
        q, scale, zero = _w4_codes(normal(N, K, scale=K ** -0.5), c)
        s["codes"][e] = q[:, 0::2] | (q[:, 1::2] << 4)
        s["scales"][e] = scale
        if c["zeros"]:
            s["zeros"][e] = zero
    return s


# ------------------------------------------------------------------ plain forms
def _scores(logits, score):
    """fp64 scores, and which experts are left out by their logits."""
    l = logits.double()
    l = torch.where(l.isnan(), -_INF, l)
    out = l == -_INF
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-l)), l, out
    m = l.amax(1, keepdim=True)
    p = torch.where(l == m, 1.0, torch.exp(l - m)).masked_fill(out, 0.0)
    total = p.sum(1, keepdim=True)
    return p / torch.where(total == 0, 1.0, total), l, out


def _plain_select(s):
    c = s["c"]
    T, E, k, n = c["T"], c["E"], c["k"], c["groups"]
    score, l, out = _scores(s["logits"], c["score"])
    choice = l  # in the scores' order
    if s["bias"] is not None:
        choice = (score + s["bias"].double()).masked_fill(out, -_INF)
    if n > 1:
        value = (score.masked_fill(out, -_INF) if s["bias"] is None else choice).view(T, n, E // n)
        best = torch.sort(value, dim=2, descending=True).values
        total = best[..., 0]
        if c["group_top"] == 2 and E // n > 1:
            total = total + torch.where(best[..., 1] == -_INF, 0.0, best[..., 1])
        kept = torch.sort(total, dim=1, descending=True, stable=True).indices[:, :c["group_k"]]
        keep = torch.zeros(T, n, dtype=torch.bool, device=l.device).scatter_(1, kept, True)
        choice = choice.masked_fill(~keep.repeat_interleave(E // n, dim=1), -_INF)
    top = torch.sort(choice, dim=1, descending=True, stable=True)
    ids, none = top.indices[:, :k], top.values[:, :k] == -_INF
    w = score.gather(1, ids).masked_fill(none, 0.0)
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total == 0, 1.0, total)
    r = dict(ids=ids.masked_fill(none, -1).to(torch.int32), w=(_SCALE * w).float())
    if c["scores"]:
        r["scores"] = score.float()
    return r


_SCALE = 2.5  # the weights' factor


def _plain_select_bwd(s):
    c = s["c"]
    score, _, _ = _scores(s["logits"], c["score"])
    none = s["ids"] < 0
    ids = s["ids"].clamp(min=0).long()
    dw, chosen = s["dw"].double().masked_fill(none, 0.0), score.gather(1, ids).masked_fill(none, 0.0)
    if c["renorm"]:
        q = chosen.sum(1, keepdim=True)
        q = torch.where(q == 0, _INF, q)
        ds = _SCALE * (dw - (dw * chosen / q).sum(1, keepdim=True)) / q
    else:
        ds = _SCALE * dw
    grad = torch.zeros_like(score) if s["dscores"] is None else s["dscores"].double()
    grad = grad.scatter_add(1, ids, ds.masked_fill(none, 0.0))
    if c["score"] == "sigmoid":
        dl = score * (1 - score) * grad
    else:
        dl = score * (grad - (score * grad).sum(1, keepdim=True))
    return dl.to(_DTYPES[c["dl"]])


def _w4_codes(x, c):
    """Codes (one byte each), scales and zero points of x [..., K] in groups along K: scales in fp32, quotients in 64
    bits (bf16 values often lie half way between two codes)."""
    v = x.float().reshape(*x.shape[:-1], -1, c["group"])
    if c["zeros"]:
        low = v.amin(-1).clamp(max=0.0)
        scale = ((v.amax(-1).clamp(min=0.0) - low) / 15).to(_DTYPES[c["sdtype"]])
    else:
        scale = (v.abs().amax(-1) / 7).to(_DTYPES[c["sdtype"]])
    step = torch.where(scale == 0, _INF, scale.double())
    if c["zeros"]:
        zero = torch.round(-low / step).clamp(0, 15)
    else:
        zero = torch.full_like(step, 8.0)
    q = (torch.round(v / step[..., None]) + zero[..., None]).clamp(0, 15)
    return q.to(torch.uint8).reshape(x.shape), scale, zero.to(torch.uint8)


def _w4_values(q, scale, zero, group):
    """fp32 values of codes (one byte each)."""
    v = q.float().reshape(*q.shape[:-1], -1, group) - (8.0 if zero is None else zero.float()[..., None])
    return (v * scale.float()[..., None]).reshape(q.shape)


def _weights(s, e=slice(None)):
    q = s["codes"][e]
    q = torch.stack((q & 15, q >> 4), dim=-1).flatten(-2)
    return _w4_values(q, s["scales"][e], None if s["zeros"] is None else s["zeros"][e], s["c"]["group"])


def _plain_product(s):
    c, M = s["c"], s["c"]["T"] * s["c"]["k"]
    off, a = s["offsets"].long(), s["a"]
    if s["index"] is not None:
        a = a[torch.div(s["index"], c["k"], rounding_mode="floor").long()]
    r = torch.arange(M, device=off.device)
    e = (off[1:, None] <= r).sum(0)
    if M <= c["E"]:  # few rows: each with its own expert's weights
        y = torch.matmul(_weights(s, e), a.float()[:, :, None])[:, :, 0]
    else:
        rows = off[:-1, None] + torch.arange(s["widest"], device=off.device)
        x = a[rows.clamp(max=M - 1)].float() * (rows < off[1:, None]).unsqueeze(-1)
        y = torch.matmul(x, _weights(s).transpose(1, 2).contiguous())[e, r - off[e]]
    return y.to(_DTYPES[c["out"]])


def _plain(s):
    c, op = s["c"], s["c"]["op"]
    if op == "select":
        return _plain_select(s)
    if op == "select_bwd":
        return _plain_select_bwd(s)
    if op == "product":
        return _plain_product(s)
    q, scale, zero = _w4_codes(s["x"].transpose(1, 2).contiguous() if c["trans"] else s["x"], c)
    r = dict(values=_w4_values(q, scale, zero, c["group"]).to(s["x"].dtype), scales=scale)
    if c["zeros"]:
        r["zeros"] = zero
    return r


# ------------------------------------------------------------------ the library's calls
def _own(s):
    import sparse_moe_layer_gemm_amd as moe
    c, op = s["c"], s["c"]["op"]

    def empty(*shape, dtype):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    if op == "select":
        ids, w = empty(c["T"], c["k"], dtype=torch.int32), empty(c["T"], c["k"], dtype=torch.float32)
        scores = empty(c["T"], c["E"], dtype=torch.float32) if c["scores"] else None
        moe.moe_select(s["logits"], ids, w, score=c["score"], bias=s["bias"], groups=c["groups"], group_k=c["group_k"],
                       group_top=c["group_top"], renorm=c["renorm"], scale=_SCALE, scores=scores)
        return dict(ids=ids, w=w, scores=scores) if c["scores"] else dict(ids=ids, w=w)
    if op == "select_bwd":
        dl = empty(c["T"], c["E"], dtype=_DTYPES[c["dl"]])
        moe.moe_select_backward(s["logits"], s["ids"], s["dw"], dl, score=c["score"], renorm=c["renorm"], scale=_SCALE,
                                dscores=s["dscores"])
        return dl
    if op == "product":
        out = empty(c["T"] * c["k"], c["N"], dtype=_DTYPES[c["out"]])
        moe.moe_w4_grouped_gemm(s["a"], s["codes"], s["scales"], s["offsets"], out, zeros=s["zeros"],
                                row_index=s["index"], row_div=c["k"] if c["gather"] else 1)
        return out
    rows, K = ((c["B"], c["C"]), c["R"]) if c["trans"] else ((c["R"],), c["C"])
    codes = empty(*rows, K // 2, dtype=torch.uint8)
    scales = empty(*rows, K // c["group"], dtype=_DTYPES[c["sdtype"]])
    zeros = empty(*rows, K // c["group"], dtype=torch.uint8) if c["zeros"] else None
    values = empty(*rows, K, dtype=s["x"].dtype)
    moe.moe_w4_quantize(s["x"], codes, scales, zeros=zeros, trans=c["trans"])
    moe.moe_w4_dequantize(codes, scales, values, zeros=zeros)
    r = dict(values=values, scales=scales)
    if c["zeros"]:
        r["zeros"] = zeros
    return r


def run(s):
    return _own(s) if own else _plain(s)


# ------------------------------------------------------------------ 64 bits
def _log_scores(l, score):
    """Logarithms of the scores, from the logits in fp64."""
    if score == "sigmoid":
        return -torch.log1p(torch.exp(-l.abs())) + l.clamp(max=0)
    return l - torch.logsumexp(l, dim=1, keepdim=True).nan_to_num(neginf=0.0)


def _exact_select(c, s):
    T, E, k, n = c["T"], c["E"], c["k"], c["groups"]
    l = s["logits"].double()
    prob = torch.exp(_log_scores(l, c["score"]))
    value = prob if s["bias"] is None else prob + s["bias"].double()
    value = torch.where(l > -_INF, value, torch.full_like(value, -1e30))
    if n > 1:
        by = value.view(T, n, -1)
        first = by.amax(2)
        if c["group_top"] == 2 and E > n:
            at = by.argmax(2, keepdim=True)
            second = by.scatter(2, at, -1e30).amax(2)
            first = first + torch.where(second < -1e29, torch.zeros_like(second), second)
        for _ in range(n - c["group_k"]):  # the worst group goes, of equally bad ones the last
            worst = n - 1 - first.flip(1).argmin(1)
            by = by.scatter(1, worst[:, None, None].expand(T, 1, E // n), -1e30)
            first = first.scatter(1, worst[:, None], _INF)
        value = by.reshape(T, E)
    ids, logw, own_value = [], [], value
    for _ in range(k):
        best = own_value.amax(1, keepdim=True)
        at = (own_value == best).to(torch.int8).argmax(1, keepdim=True)
        none = best < -1e29
        ids.append(torch.where(none, -torch.ones_like(at), at))
        logw.append(torch.where(none, torch.full_like(best, -_INF), _log_scores(l, c["score"]).gather(1, at)))
        own_value = own_value.scatter(1, at, -1e30)
    ids, logw = torch.cat(ids, 1), torch.cat(logw, 1)
    w = torch.softmax(logw, 1).nan_to_num(0.0) if c["renorm"] else torch.exp(logw)
    r = dict(ids=ids.to(torch.int32), w=2.5 * w)
    if c["scores"]:
        r["scores"] = prob
    return r


def _exact_select_bwd(c, s):
    """Gradients from the logarithms of the scores: d s = s d(log s)."""
    l, ids = s["logits"].double(), s["ids"].long()
    logs = _log_scores(l, c["score"])
    ok = ids >= 0
    logc = torch.where(ok, logs.gather(1, ids.clamp(min=0)), torch.full_like(s["dw"].double(), -_INF))
    dw = 2.5 * s["dw"].double() * ok
    if c["renorm"]:
        r = torch.softmax(logc, 1).nan_to_num(0.0)
        dlog = r * (dw - (r * dw).sum(1, keepdim=True))
    else:
        dlog = torch.exp(logc) * dw
    d = torch.zeros_like(l)
    for j in range(c["k"]):
        d.scatter_add_(1, ids[:, j:j + 1].clamp(min=0), dlog[:, j:j + 1] * ok[:, j:j + 1])
    prob = torch.exp(logs)
    if s["dscores"] is not None:
        d = d + prob * s["dscores"].double()
    if c["score"] == "sigmoid":
        return d * torch.exp(_log_scores(-l, "sigmoid"))
    return d - prob * d.sum(1, keepdim=True)


def _exact_weights(s, e):
    c, q = s["c"], s["codes"][e].long()
    q = torch.stack((q % 16, q // 16), dim=-1).flatten(-2).double()
    z = 8.0 if s["zeros"] is None else s["zeros"][e].double().repeat_interleave(c["group"], dim=-1)
    return (q - z) * s["scales"][e].double().repeat_interleave(c["group"], dim=-1)


def _nearest(x):
    """The nearest whole number, of two equally near ones the even one."""
    low = torch.floor(x)
    up = (x - low > 0.5) | ((x - low == 0.5) & (low.remainder(2) == 1))
    return low + up


def exact(case, seed):
    s = prepare(case, seed)
    c, op = s["c"], s["c"]["op"]
    if op == "select":
        return _exact_select(c, s)
    if op == "select_bwd":
        return _exact_select_bwd(c, s)
    if op == "product":
        M, off = c["T"] * c["k"], s["offsets"].tolist()
        out = torch.zeros(M, c["N"], dtype=torch.float64, device="cuda")
        source = torch.arange(M, device="cuda") if s["index"] is None else s["index"].long() // c["k"]
        for e in range(c["E"]):
            if off[e] < off[e + 1]:
                rows = source[off[e]:off[e + 1]]
                out[off[e]:off[e + 1]] = s["a"][rows].double() @ _exact_weights(s, e).t().contiguous()
        return out
    x = s["x"] if c["trans"] else s["x"][None]
    values, scales, zeros = [], [], []
    for part in x:
        v = (part.t().contiguous() if c["trans"] else part).double()
        v = v.reshape(v.shape[0], -1, c["group"])
        top, low = v.amax(-1).clamp(min=0), v.amin(-1).clamp(max=0)
        # the scale is fp32 arithmetic rounded to its own type, as the format has it
        step = (top.float() - low.float()) / 15 if c["zeros"] else torch.maximum(top, -low).float() / 7
        step = step.to(_DTYPES[c["sdtype"]])
        d = step.double()
        z = _nearest(-low / d) if c["zeros"] else torch.full_like(d, 8.0)
        q = _nearest(v / d[..., None])
        q = torch.minimum(torch.maximum(q, -z[..., None]), 15 - z[..., None])
        values.append((q * d[..., None]).flatten(1))
        scales.append(step)
        zeros.append(z.to(torch.uint8))
    r = dict(values=torch.stack(values) if c["trans"] else values[0], scales=torch.stack(scales) if c["trans"] else scales[0])
    if c["zeros"]:
        r["zeros"] = torch.stack(zeros) if c["trans"] else zeros[0]
    return r
