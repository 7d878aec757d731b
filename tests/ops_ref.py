"""Plain 64-bit forms of the grouped products, SwiGLU, the finalize gradient and
MXFP4, and helpers that place tensors between guard values."""
import torch

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step of each type


def offsets_of(counts, device="cuda"):
    off = [0]
    for c in counts:
        off.append(off[-1] + c)
    return torch.tensor(off, dtype=torch.int32, device=device)


def guarded(t, pad, value):
    """t's values inside a larger buffer: `pad` elements of `value` on both sides (pad a multiple of 16)."""
    big = torch.full((t.numel() + 2 * pad,), value, dtype=t.dtype, device=t.device)
    view = big[pad:pad + t.numel()].view(t.shape)
    view.copy_(t)
    return view, big


def guards_intact(big, pad, value):
    edge = torch.cat((big[:pad], big[big.numel() - pad:]))
    return bool((edge == value).all())


def gather64(a, M, row_index=None, row_div=1):
    if row_index is None:
        return a[:M].double()
    s = torch.div(row_index.long(), row_div, rounding_mode="floor")
    ok = (row_index >= 0) & (s < a.shape[0])
    x = a[s.clamp(0, a.shape[0] - 1)].double()
    return torch.where(ok[:, None], x, torch.zeros_like(x))


def product64(x, w, counts, w_trans):
    """(rows of the product, sum of |terms|) for gathered fp64 rows x."""
    n = w.shape[1] if w_trans else w.shape[2]
    out = torch.zeros(sum(counts), n, dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(out)
    lo = 0
    for e, c in enumerate(counts):
        if c:
            we = w[e].double().t().contiguous() if w_trans else w[e].double()
            out[lo:lo + c] = x[lo:lo + c] @ we
            mag[lo:lo + c] = x[lo:lo + c].abs() @ we.abs()
        lo += c
    return out, mag


def wgrad64(x, d, counts):
    out = torch.zeros(len(counts), x.shape[1], d.shape[1], dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(out)
    lo = 0
    for e, c in enumerate(counts):
        if c:
            xe, de = x[lo:lo + c].t().contiguous(), d[lo:lo + c].double()
            out[e], mag[e] = xe @ de, xe.abs() @ de.abs()
        lo += c
    return out, mag


def sum_bound(ref, mag, depth, dtype):
    """Largest |error| of a sum of `depth` exact products in fp32, rounded once to dtype: every
    addition is off by at most one step (2^-23) of a partial sum no larger than mag."""
    acc = depth * 2.0 ** -23 * mag
    return acc + HALF[dtype] * (ref.abs() + acc)


def two_to(e):
    """2^e in fp64 for whole numbers e, from its bits (torch's pow is not exact on every power of two)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def mx_decode64(codes, scales):
    nib = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).long()
    grid = torch.tensor(GRID + tuple(-v for v in GRID), dtype=torch.float64, device=codes.device)
    b = scales[..., : nib.shape[-1] // 32].double()
    step = torch.where(b == 255, torch.full_like(b, float("nan")), two_to(b - 127))
    return grid[nib] * step.repeat_interleave(32, dim=-1)


def mx_encode(x):
    """(codes one byte each, scale bytes) of x [..., K] in fp64 arithmetic."""
    b = x.double().reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    top = b.abs().amax(-1, keepdim=True)
    bad = ~torch.isfinite(b).all(-1, keepdim=True)
    top = torch.where(bad, torch.ones_like(top), top)
    # floor(log2): frexp gives top = f * 2^e with f in [1/2, 1)
    e = (torch.frexp(top).exponent.double() - 3).clamp(min=-127)
    e = torch.where(top == 0, torch.full_like(e, -127.0), e)
    q = b * two_to(-e)
    grid = torch.tensor(GRID, dtype=torch.float64, device=x.device)
    dist = (q.abs().unsqueeze(-1) - grid).abs()
    odd = torch.arange(8, device=x.device) % 2
    near = dist == dist.amin(-1, keepdim=True)  # ties: the even code
    code = torch.where(near, odd, torch.full_like(odd, 2)).argmin(-1)
    code = code + 8 * torch.signbit(b).long()
    code = torch.where(bad, torch.zeros_like(code), code)
    scale = torch.where(bad, torch.full_like(e, 255.0), e + 127)
    return code.reshape(x.shape).to(torch.uint8), scale.squeeze(-1).to(torch.uint8)


def mx_pack(code):
    return (code[..., 0::2] | (code[..., 1::2] << 4)).contiguous()
