"""Shared pieces of the norm, gate and 8-bit storage tests: seeded inputs,
guarded outputs and the rounding steps tolerances are counted in."""
import numpy as np
import torch

import fp4_spectral_split_amd as M

U32 = 2.0 ** -24  # half a step of fp32, relative
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
T = {"f32": torch.float32, "bf16": torch.bfloat16}


def np64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def to_dev(x, dtype, pad=0, shift=0):
    """x on the GPU as a view whose rows are pad elements longer and start
    shift elements into their buffer."""
    rows, cols = x.shape
    buf = torch.zeros(rows * (cols + pad) + shift, dtype=dtype, device="cuda")
    v = buf[shift:].view(rows, cols + pad)[:, :cols]
    v.copy_(torch.from_numpy(np.ascontiguousarray(x)).to(dtype))
    return v


class Guard:
    """An output tensor inside a sentinel-filled buffer, with a row pad."""

    def __init__(self, rows, cols, dtype, pad=0, shift=0):
        esz = torch.empty(0, dtype=dtype).element_size()
        self.raw = torch.full((256 + (rows * (cols + pad) + shift) * esz + 256,), 0xA5, dtype=torch.uint8,
                              device="cuda")
        self.at, self.n, self.esz = 256 + shift * esz, rows * (cols + pad), esz
        self.rows, self.cols, self.pad = rows, cols, pad
        self.t = self.raw[self.at:self.at + self.n * esz].view(dtype).view(rows, cols + pad)[:, :cols]

    def intact(self):
        r = self.raw.cpu().numpy()
        body = r[self.at:self.at + self.n * self.esz].reshape(self.rows, -1)[:, self.cols * self.esz:]
        return bool(np.all(r[:self.at] == 0xA5) and np.all(r[self.at + self.n * self.esz:] == 0xA5)
                    and np.all(body == 0xA5))


def guarded_act8(fmt, rows, cols):
    """An Act8Tensor in guarded buffers, the codes at an odd address."""
    c = Guard(1, rows * cols, torch.uint8, shift=1)
    s = Guard(1, rows * -(-cols // 32), torch.uint8, shift=1)
    return M.Act8Tensor(M._FMT8[fmt], rows, cols, c.t.view(-1), s.t.view(-1)), (c, s)


def act8_np(q):
    return (q.codes.cpu().numpy().reshape(q.rows, q.cols), q.scales.cpu().numpy().reshape(q.rows, -1))
