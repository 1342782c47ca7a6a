"""Plain 64-bit forms of MXFP4 values and products, for the tests of the products and gradients."""
import torch

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def value(q, s):
    """Codes [..., K/2] and scale bytes [..., K/32] -> float64 [..., K]."""
    table = torch.tensor(GRID + tuple(-g for g in GRID), dtype=torch.float64, device=q.device)
    v = table[torch.stack([q & 15, q >> 4], -1).flatten(-2).long()]
    # 2^(s - 127) by its bits: a device's pow need not be exact
    scale = ((s.long() + (1023 - 127)) << 52).view(torch.float64)
    return v * torch.where(s == 255, float("nan"), scale).repeat_interleave(32, -1)


def random_mx(gen, shape, spread=6):
    """Codes of every kind and scales over 2 * spread + 1 binades around 1."""
    dev = gen.device
    K = shape[-1]
    q = torch.randint(0, 256, shape[:-1] + (K // 2,), generator=gen, device=dev, dtype=torch.uint8)
    s = torch.randint(127 - spread, 128 + spread, shape[:-1] + (K // 32,), generator=gen, device=dev,
                      dtype=torch.uint8)
    return q, s


def product_bound(absolute, K, alpha, dtype, result):
    """|error| allowed to a product of K terms: each fp32 addition, truncating or rounding, is off by
    less than one step (2^-23) of a running sum that never exceeds the sum of the magnitudes
    ``absolute``; alpha's multiplication and the rounding to the output type add half a step each."""
    half = torch.finfo(dtype).eps / 2
    acc = K * 2.0 ** -23 * absolute * abs(alpha)
    return acc + (half + 2.0 ** -24) * (result.abs() + acc) + 1e-37


def guarded(shape, dtype, device, fill):
    """A buffer of ``shape`` with 1024 elements behind it, all holding ``fill``: (view, whole)."""
    n = 1
    for d in shape:
        n *= d
    whole = torch.full((n + 1024,), fill, dtype=dtype, device=device)
    return whole[:n].view(shape), whole


def behind_untouched(view, whole, fill):
    return bool((whole[view.numel():] == fill).all())
