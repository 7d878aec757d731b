"""Plain 64-bit forms of 4-bit integer weights with group scales."""
import torch

INF = float("inf")


def quantise(x, group, zeros, sdtype):
    """(codes one byte each, scales, zero points or None) of x [..., K]: scales in fp32, quotients in 64 bits."""
    v = x.float().reshape(*x.shape[:-1], -1, group)
    bad = ~torch.isfinite(v).all(-1)
    v = torch.where(bad[..., None], torch.zeros_like(v), v)
    if zeros:
        low = v.amin(-1).clamp(max=0.0)
        s = (v.amax(-1).clamp(min=0.0) - low) * torch.tensor(1 / 15, dtype=torch.float32, device=v.device)
    else:
        s = v.abs().amax(-1) * torch.tensor(1 / 7, dtype=torch.float32, device=v.device)
    bad = bad | ~torch.isfinite(s)
    s = s.to(sdtype)
    step = torch.where((s == 0) | bad, INF, s.double())
    z = torch.round(-low.double() / step).clamp(0, 15) if zeros else torch.full_like(step, 8.0)
    q = (torch.round(v.double() / step[..., None]) + z[..., None]).clamp(0, 15)
    s = torch.where(bad, torch.full_like(s, float("nan")), s)
    return q.to(torch.uint8).reshape(x.shape), s, z.to(torch.uint8) if zeros else None


def pack(q):
    return (q[..., 0::2] | (q[..., 1::2] << 4)).contiguous()


def unpack(codes):
    return torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2)


def weights64(codes, scales, zeros=None):
    q = unpack(codes).double()
    group = q.shape[-1] // scales.shape[-1]
    z = 8.0 if zeros is None else zeros.double().repeat_interleave(group, dim=-1)
    return (q - z) * scales.double().repeat_interleave(group, dim=-1)


def spread64(codes, scales, zeros=None):
    """(q + z) |s|, what a product's fp32 sums run over: the codes and the zero points are summed apart."""
    q = unpack(codes).double()
    group = q.shape[-1] // scales.shape[-1]
    z = 8.0 if zeros is None else zeros.double().repeat_interleave(group, dim=-1)
    return (q + z) * scales.double().abs().repeat_interleave(group, dim=-1)
