"""Helpers of the row-wise calls' GPU tests: inputs inside marked buffers, and
comparison with fp64 results within bounds."""
import torch

F32, BF16 = torch.float32, torch.bfloat16
U = 2.0 ** -24                     # half a step of fp32, relative
HALF = {F32: U, BF16: 2.0 ** -8}
MARK = 7.0


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(shape, std, seed, dtype=F32, mean=0.0):
    return (torch.randn(shape, generator=gen(seed)) * std + mean).to(dtype)


class Placed:
    """Rows on the GPU inside a buffer of marks: `pad` elements between them, the first `shift` elements in."""

    def __init__(self, x, pad=0, shift=0):
        rows, cols = x.shape
        self.buffer = torch.full((shift + rows * (cols + pad) + 8,), MARK, device="cuda", dtype=x.dtype)
        self.view = self.buffer[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
        self.view.copy_(x)
        self.at = (rows, cols, pad, shift)

    def untouched(self):
        rows, cols, pad, shift = self.at
        own = torch.zeros(self.buffer.numel(), dtype=torch.bool, device="cuda")
        own[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols] = True
        return bool((self.buffer[~own] == MARK).all())


def close(got, want, bound, what, dtype=None):
    """Within `bound` (fp64), and half a step of the stored type where it is not fp32."""
    dtype = dtype or got.dtype
    got = got.detach().float().cpu().double()
    assert got.shape == want.shape, f"{what}: shape {tuple(got.shape)}"
    if dtype == BF16:
        bound = bound + HALF[BF16] * (want.abs() + bound)
    bad = ~((got - want).abs() <= bound)
    bad &= ~((got == want) | (got.isnan() & want.isnan()))
    if bad.any():
        i = int(bad.flatten().nonzero()[0])
        worst = ((got - want).abs() / bound.expand_as(want)).flatten()[bad.flatten()].max()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} beyond the bound, worst {worst:.3g} times; first at {i}: "
                             f"{got.flatten()[i]:.9g}, not {want.flatten()[i]:.9g}")
