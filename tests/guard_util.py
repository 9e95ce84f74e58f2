"""Tensors inside larger buffers, to see reads and writes beside them."""
import torch

PAD = 1 << 20  # bytes in front and behind, more than the rows of a tile of the tests' sizes
BYTE = 0xA5


class Guards:
    """Tensors between bytes that nothing may write.  `offset`: elements behind an aligned address."""

    def __init__(self):
        self.kept = []

    def _place(self, nbytes, at):
        raw = torch.full((nbytes + at + 2 * PAD,), BYTE, dtype=torch.uint8, device="cuda")
        self.kept.append((raw, PAD + at, nbytes))
        return raw[PAD + at:PAD + at + nbytes]

    def output(self, shape, dtype, offset=0):
        size = torch.empty((), dtype=dtype).element_size()
        n = 1
        for q in shape:
            n *= q
        return self._place(n * size, offset * size).view(dtype).view(shape)

    def workspace(self, nbytes):
        """Of exactly as many bytes, which hold NaNs of every type."""
        return self._place(nbytes, 0).fill_(255)

    def assert_whole(self):
        for i, (raw, at, n) in enumerate(self.kept):
            assert bool((raw[:at] == BYTE).all()), "buffer %d, in front" % i
            assert bool((raw[at + n:] == BYTE).all()), "buffer %d, behind" % i


def among_nan(t, offset=0):
    """A copy of t between NaNs: what is read beside it shows in the results."""
    pad = PAD // t.element_size()
    raw = torch.full((t.numel() + offset + 2 * pad,), float("nan"), dtype=t.dtype, device="cuda")
    return raw[pad + offset:pad + offset + t.numel()].view(t.shape).copy_(t)
