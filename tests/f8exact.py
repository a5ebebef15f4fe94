"""Operands of the e4m3 products whose sums every form has to give exactly: small integers and
scales of one and two, so that products, block sums and scaled sums are integers far below 2^24 (and
what the 8-bit matrix cores drop, below 2^-13 of the largest of eight products, is nothing)."""
from __future__ import annotations

import torch

DEV = "cuda:0"
F8 = torch.float8_e4m3fn
VALUES = [-2.0, -1.0, 0.0, 0.0, 0.0, 0.0, 1.0, 2.0]
CODES = [0xC0, 0xB8, 0x00, 0x00, 0x00, 0x00, 0x38, 0x40]


def units():
    return torch.cuda.get_device_properties(0).multi_processor_count


def up(n, m):
    return -(-n // m) * m


class Operands:
    """Weights of E matrices (M, K) and X rows, with their exact values in float64."""

    def __init__(self, E, M, K, X, seed, bias):
        g = torch.Generator(device=DEV).manual_seed(seed)
        table, values = torch.tensor(CODES, dtype=torch.uint8, device=DEV), torch.tensor(VALUES, dtype=torch.float64, device=DEV)
        nb = -(-K // 128)

        def draw(*shape):
            return torch.randint(0, 8, shape, generator=g, device=DEV)

        def scales(*shape):
            return torch.randint(1, 3, shape, generator=g, device=DEV).float()

        wi, xi = draw(E, M, K), draw(X, K)
        self.E, self.M, self.K, self.X = E, M, K, X
        self.w, self.ws = table[wi].view(F8), scales(E, -(-M // 128), nb)
        xq = torch.zeros(X, nb * 128, dtype=torch.uint8, device=DEV)
        xq[:, :K] = table[xi]
        self.xq = xq.view(F8)
        xs = scales(X, nb)
        self.xs = torch.full((X, up(nb, 4)), float("nan"), device=DEV)  # what lies beyond the blocks may be anything
        self.xs[:, :nb] = xs
        self.bias = torch.randint(-9, 10, (E, M), generator=g, device=DEV).float() if bias else None
        self.wv = values[wi] * self.ws.double().repeat_interleave(128, 1)[:, :M].repeat_interleave(128, 2)[:, :, :K]
        self.xv = values[xi] * xs.double().repeat_interleave(128, 1)[:, :K]

    def product(self, e, rows, dtype):
        """The product of rows of x (a slice or indices) with matrix e, rounded once."""
        y = torch.mm(self.xv[rows], self.wv[e].t().contiguous())
        return (y if self.bias is None else y + self.bias[e].double()).to(dtype)
