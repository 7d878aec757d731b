"""Plain 64-bit forms of routing by scores and its gradient, one token at a time in Python numbers."""
import math
import struct

import torch

INF = float("inf")


def _sig(l):
    return 1 / (1 + math.exp(-l)) if l >= -700 else math.exp(l) if l > -INF else 0.0


def _one_minus_sig(l):
    return _sig(-l) if l < INF else 0.0


def bits44(x):
    """x without the last 8 of its 52 fraction bits: what choices with a bias are compared by."""
    return struct.unpack("d", struct.pack("Q", struct.unpack("Q", struct.pack("d", x))[0] & ~255))[0]


def scores_of(logits, score):
    """Scores of one token (a list): NaN counts as -infinity, +infinity as the limit of large numbers."""
    l = [-INF if x != x else x for x in logits]
    if score == "sigmoid":
        return [_sig(x) for x in l]
    m = max(l)
    if m == -INF:
        return [0.0] * len(l)
    e = [1.0 if x == m else math.exp(x - m) for x in l]
    total = math.fsum(e)
    return [x / total for x in e]


def select(logits, k, score="softmax", bias=None, groups=1, group_k=1, group_top=1, renorm=True, scale=1.0):
    """(ids [T, k], weights [T, k] fp64, scores [T, E] fp64) of logits [T, E]."""
    ids, ws, ss = [], [], []
    E = logits.shape[1]
    for row in logits.double().tolist():
        s = scores_of(row, score)
        may = [x == x and x != -INF for x in row]
        choice = list(row)
        if bias is not None:
            b = bias.double().tolist()
            may = [m and x == x and x != -INF for m, x in zip(may, b)]
            choice = [bits44(x + y) if x + y == x + y else x + y for x, y in zip(s, b)]
        left = [e for e in range(E) if may[e]]
        if groups > 1:
            size, value = E // groups, {}
            for g in range(groups):
                own = sorted((choice[e] for e in left if e // size == g), reverse=True)
                if own and group_top == 1:
                    value[g] = own[0]
                elif own:
                    own = own if bias is not None else sorted((s[e] for e in left if e // size == g), reverse=True)
                    value[g] = sum(own[:2])
            kept = sorted(value, key=lambda g: (-value[g], g))[:group_k]
            left = [e for e in left if e // size in kept]
        top = sorted(left, key=lambda e: (-choice[e], e))[:k]
        w = [s[e] for e in top]
        if renorm and score == "softmax" and top:  # as a softmax over the chosen: no underflow
            w = scores_of([row[e] for e in top], "softmax")
        elif renorm:
            total = math.fsum(w)
            w = [x / total if total else 0.0 for x in w]
        ids.append(top + [-1] * (k - len(top)))
        ws.append([scale * x for x in w] + [0.0] * (k - len(top)))
        ss.append(s)
    return torch.tensor(ids, dtype=torch.int32), torch.tensor(ws, dtype=torch.float64), torch.tensor(ss, dtype=torch.float64)


def backward(logits, ids, dw, score="softmax", renorm=True, scale=1.0, dscores=None):
    """(d logits [T, E], a bound of their error before the last rounding) in fp64, from the formula.

    The bound counts fp32 roundings of 2^-24: a slot's part is rounded once and added at most 8 times; the dense part
    needs, per expert, an exponential (2, and |x - m| for its argument's rounding), sums of 16 + 4 terms, a quotient
    and a handful of products, each on a magnitude of at most s (|g| + sum |s g| + sum |c|).
    """
    T, E = logits.shape
    out, bound = [], []
    u = 2.0 ** -24
    for t, row in enumerate(logits.double().tolist()):
        s = scores_of(row, score)
        part, mag = [0.0] * E, [0.0] * E
        slots = [(e, d) for e, d in zip(ids[t].tolist(), dw[t].double().tolist())
                 if 0 <= e < E and row[e] == row[e] and row[e] != -INF]
        # r: renormalised scores of the slots
        if renorm:
            if score == "softmax":
                r = scores_of([row[e] for e, _ in slots], "softmax") if slots else []
            else:
                total = math.fsum(s[e] for e, _ in slots)
                r = [s[e] / total if total else 0.0 for e, _ in slots]
            mean = math.fsum(d * x for (_, d), x in zip(slots, r))
        else:
            r, mean = [s[e] for e, _ in slots], 0.0
        spread = 0.0
        for (e, d), x in zip(slots, r):
            c = scale * x * (d - mean) * (_one_minus_sig(row[e]) if score == "sigmoid" else 1.0)
            part[e] += c
            mag[e] += abs(c)
            spread += c
        g = dscores[t].double().tolist() if dscores is not None else [0.0] * E
        if score == "softmax":
            total = math.fsum(x * y for x, y in zip(s, g) if x) + (0.0 if renorm else spread)
            size = math.fsum(abs(x * y) for x, y in zip(s, g) if x) + (0.0 if renorm else sum(mag))
            dense = [x * (y - total) if x else 0.0 for x, y in zip(s, g)]
            finite = [x for x in row if abs(x) < INF]
            far = max([0.0] + [min(max(finite) - x, 104.0) for x in finite])
            err = [2 * u * (far + 80) * x * (abs(y) + 2 * size) if x else 0.0 for x, y in zip(s, g)]
            if not (dscores is not None or not renorm):
                dense, err = [0.0] * E, [0.0] * E
        else:
            dense = [x * _one_minus_sig(l) * y if x else 0.0 for x, y, l in zip(s, g, row)]
            err = [12 * u * abs(x) for x in dense]
        out.append([p + d for p, d in zip(part, dense)])
        bound.append([e + 10 * u * m + u * abs(p + d) + 1e-37 for e, m, p, d in zip(err, mag, part, dense)])
    return torch.tensor(out, dtype=torch.float64).view(T, E), torch.tensor(bound, dtype=torch.float64).view(T, E)


def backward_sure(logits, ids, dw, score, renorm, scale, dscores=None):
    """(d logits, a bound of their error) as backward's, by sums over pairs of experts: d - sum d r is sum_i r_i (d_j - d_i), which
    loses nothing where one expert has nearly all of the sum. Rows without infinities, ids that differ.

    The bound counts fp32 roundings, u = 2^-24. Softmax: s is off by |x - m| + 36, the moved h (h less that of the expert that
    has more than half, formed from the parts of both) by 3, its products with s, their sum and the last difference and product
    by 26: K = |x - m| + 50 for every s, of what is moved. What the slots give besides: 1 of itself, and fp64 roundings."""
    u = 2.0 ** -24
    T, E = logits.shape
    out, bound = [], []
    for t, row in enumerate(logits.double().tolist()):
        s = scores_of(row, score)
        slots = list(zip(ids[t].tolist(), dw[t].double().tolist()))
        g = dscores[t].double().tolist() if dscores is not None else [0.0] * E
        dl, err, D = [0.0] * E, [0.0] * E, [0.0] * E
        if score == "softmax" and not renorm:
            for e, d in slots:
                D[e] = scale * d
        else:
            r = scores_of([row[e] for e, _ in slots], "softmax") if score == "softmax" else [s[e] for e, _ in slots]
            total = math.fsum(r) if renorm else 1.0
            r = [x / total for x in r]
            for (e, d), x in zip(slots, r):
                w = scale * x * (_one_minus_sig(row[e]) if score == "sigmoid" else 1.0)
                terms = [y * (d - c) for (_, c), y in zip(slots, r)] if renorm else [d]
                dl[e] = w * math.fsum(terms)
                err[e] = 1.01 * u * abs(dl[e]) + 2.0 ** -44 * abs(w) * sum(abs(v) for v in terms)
        if score == "sigmoid":
            for e in range(E):
                v = s[e] * _one_minus_sig(row[e]) * g[e]
                err[e] += 12 * u * abs(v) + u * abs(dl[e] + v)
                dl[e] += v
        elif dscores is not None or not renorm:
            most = max(range(E), key=lambda e: s[e])
            d0, g0 = (D[most], g[most]) if s[most] > 0.5 else (0.0, 0.0)
            H = [abs(D[e] - d0) + abs(g[e] - g0) for e in range(E)]
            K = [max(row) - x + 50 for x in row]
            for e in range(E):
                v = s[e] * math.fsum(s[f] * ((D[e] - D[f]) + (g[e] - g[f])) for f in range(E))
                err[e] += u * s[e] * (K[e] * H[e] + math.fsum(s[f] * H[f] * (K[e] + K[f]) for f in range(E))) + u * abs(dl[e] + v)
                dl[e] += v
        out.append(dl)
        bound.append([x + 1e-37 for x in err])
    return torch.tensor(out, dtype=torch.float64).view(T, E), torch.tensor(bound, dtype=torch.float64).view(T, E)


def gradient_chain(y, dout, pos, dw, logits, ids, dl, dscores, score, renorm=True, scale=1.0):
    """A run's gradients of the weights and of the logits, each from what the step before it wrote: the largest error of
    dw [T, k] over its bound, of dl [T, E] (fp32) over its bound, and the norm of dl's bound over that of the part of dl
    that comes through the weights (what the second ratio can tell of it).

    dw: dout . y of the slot's row (pos, -1 none) in 64 bits; H products, each off by half a step of fp32, and H sums by a
    step of what they run over. dl: backward() of the dw that was written, with its bound, and dl's own rounding."""
    H = y.shape[1]
    rows = torch.where(pos[..., None] >= 0, y.double()[pos.long().clamp(min=0)], 0.0) * dout.double()[:, None]
    err = (dw.double() - rows.sum(2)).abs()
    first = (err / (2 * H * 2.0 ** -23 * rows.abs().sum(2) + 1e-37)).max().item()
    want, bound = backward(logits, ids, dw, score, renorm, scale, dscores)
    without, _ = backward(logits, ids, torch.zeros_like(dw), score, renorm, scale, dscores)
    bound = bound + 2.0 ** -24 * (want.abs() + bound)
    second = ((dl.double() - want).abs() / bound).max().item()
    return first, second, (bound.norm() / (want - without).norm()).item()
