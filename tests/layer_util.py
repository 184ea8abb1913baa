"""Inputs, 64-bit references and tolerances of the tests of the products with an epilogue,
the routing and the experts' products.

Inputs of the products are small multiples of 1/8 or 1/16, so every sum of products is exact
in fp32 and the only differences from the 64-bit reference are those of the activation and
of the one rounding to 16 bits.  A rounding is off by at most half a step, finfo.eps / 2
relative (or half of the smallest subnormal); the activations' fp32 forms are within
ACT_ERROR relative (the erfc polynomial 5.3e-6, each exp2 and reciprocal one unit in the
last place, the exponent's rounding at most |x| 2^-24 for |x| < 40)."""
import math

import torch

ACT_NONE, ACT_RELU, ACT_GELU, ACT_GELU_TANH, ACT_SILU = range(5)
ACTS = (ACT_NONE, ACT_RELU, ACT_GELU, ACT_GELU_TANH, ACT_SILU)
ACT_ERROR = 1e-5
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def eighths(shape, seed, dtype, top=8, step=8):
    """Seeded integers -top..top over `step`, on the CPU."""
    g = torch.Generator().manual_seed(seed)
    return (torch.randint(-top, top + 1, shape, generator=g).double() / step).to(dtype)


def padded(t, pad=0, offset=0, poison=float("nan")):
    """t on the GPU as rows of a wider, poisoned buffer (pad more columns, starting `offset`
    elements in): a view, and the buffer."""
    *lead, cols = t.shape
    rows = math.prod(lead)
    buf = torch.full((rows * (cols + pad) + offset + 8,), poison, dtype=t.dtype, device="cuda")
    view = buf[offset:offset + rows * (cols + pad)].view(*lead, cols + pad)[..., :cols]
    view.copy_(t)
    return view, buf


def phi(z):
    """The normal distribution function, to full relative precision below zero as well
    (torch.special.ndtr is zero from -8.3 down, where the function is not)."""
    return torch.special.erfc(-z / math.sqrt(2)) / 2


def act(kind, z):
    if kind == ACT_RELU:
        return z.clamp(min=0)
    if kind == ACT_GELU:
        return z * phi(z)
    if kind == ACT_GELU_TANH:
        return z * torch.sigmoid(math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3))
    if kind == ACT_SILU:
        return z * torch.sigmoid(z)
    return z


def act_slope(kind, z):
    if kind == ACT_RELU:
        return (z > 0).to(z.dtype)
    if kind == ACT_GELU:
        return phi(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if kind == ACT_GELU_TANH:
        c = math.sqrt(8 / math.pi)
        p = torch.sigmoid(c * (z + 0.044715 * z ** 3))
        return p + z * p * (1 - p) * c * (1 + 3 * 0.044715 * z * z)
    if kind == ACT_SILU:
        p = torch.sigmoid(z)
        return p + z * p * (1 - p)
    return torch.ones_like(z)


def layer(z, kind, gated, residual=None):
    if gated:
        h = z.shape[1] // 2
        y = act(kind, z[:, :h]) * z[:, h:]
    else:
        y = act(kind, z)
    return y if residual is None else y + residual


def layer_slope(z, dy, kind, gated):
    if not gated:
        return dy * act_slope(kind, z)
    h = z.shape[1] // 2
    return torch.cat([dy * z[:, h:] * act_slope(kind, z[:, :h]), dy * act(kind, z[:, :h])], 1)


def half_step(dtype, want):
    """Half a step of `dtype` at each value: the most that one rounding changes it."""
    info = torch.finfo(dtype)
    return (info.eps / 2) * want.abs() + info.smallest_normal * info.eps / 2


def assert_within(got, want, tol, what):
    got, want = got.double().cpu(), want.double().cpu()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    bad = ~((got - want).abs() <= tol.cpu())
    if bad.any():
        i = tuple(int(x) for x in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: "
                             f"got {got[i]}, want {want[i]}, tolerance {tol.cpu()[i]}")


def check_layer(got, z, kind, gated, residual, what):
    """C against the 64-bit epilogue of the exact z: the activation's error, two fp32
    roundings (product with the gate, residual) and the rounding of C."""
    y = layer(z, kind, gated)
    want = y if residual is None else y + residual
    # gelu below -6: the kernel's Phi(-a) follows its own fall-off there, and a Phi(-a) times
    # its relative error (3.4e-5 at 6.5, 3.9e-4 at 7, 1.9e-3 at 7.5, 4e-2 at 9, 1 past 13) is
    # below 1e-14 everywhere
    far = 1e-14 * (z[:, z.shape[1] // 2:].abs() if gated else 1.0) if kind == ACT_GELU else 0.0
    # |z| below 2^-20 cannot occur (multiples of 1/128), so the activation's relative bound
    # holds; where it has decayed below 1e-30 the fp32 form may flush
    inner = (0 if kind in (ACT_NONE, ACT_RELU) else ACT_ERROR) * y.abs() + 1e-30
    inner = inner + far + 2.0 ** -23 * (y.abs() + want.abs())
    assert_within(got, want, half_step(got.dtype, want) + 1.01 * inner, what)
