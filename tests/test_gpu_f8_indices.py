"""Grouped products with offsets and rows out of range, in every form: nothing around Y is written,
and the rows whose offsets and indices are in range are right."""
import pytest
import torch

import quantized_gemv_argmax_amd as qg
from tests.f8exact import DEV, Operands, up
from tests.gpu_helpers import case

pytestmark = pytest.mark.gpu


# streamed; tiles of 64, of 128 x 64, of 128; 256 x 128 and 256 x 256 in turns, with more tiles than units
@pytest.mark.parametrize("E,M,K,each,dtype", [(4, 96, 256, 3, torch.float32), (64, 320, 256, 2, torch.bfloat16), (4, 96, 300, 40, torch.float16),
                                              (4, 200, 640, 100, torch.float32), (4, 200, 640, 100, torch.bfloat16),
                                              (20, 2100, 512, 200, torch.float16), (4, 200, 640, 600, torch.bfloat16),
                                              (8, 2300, 512, 900, torch.float16)])
def test_grouped_indices_out_of_range(E, M, K, each, dtype):
    R, X = E * each, 50
    o = Operands(E, M, K, X, E + M, False)
    g = torch.Generator(device=DEV).manual_seed(R)
    row = torch.randint(0, X, (R,), generator=g, device=DEV, dtype=torch.int32)
    bad = torch.randint(0, R, (max(3, R // 9),), generator=g, device=DEV)
    row[bad[0::3]], row[bad[1::3]], row[bad[2::3]] = -5, X + 1000, (1 << 31) - 1
    fine = (row >= 0) & (row < X)
    w = qg.pack_f8(o.w)
    even = [e * each for e in range(E + 1)]
    for what, offsets, last in [("rows", even, E), ("beyond", even[:-2] + [R + 500, (1 << 31) - 1], E - 1), ("below", [-(1 << 31)] + even[1:], E),
                                ("descending", [-9] + even[1:-2] + [even[-2] - each - each // 2, R], 0),
                                ("all of it", [R] * E + [0], 0), ("back and forth", [0, R] * (E // 2) + [R], 0)]:
        case(f"qgemm_f8_grouped {what} E={E} M={M} K={K} each={each} {dtype}")
        whole = torch.full((R + 2, up(M, 8) + 8), -7.0, dtype=dtype, device=DEV)
        qg.qgemm_f8_grouped(w, o.ws, o.xq, o.xs, M, K, torch.tensor(offsets, dtype=torch.int64).to(torch.int32).to(DEV), row=row, Y=whole[1:-1])
        torch.cuda.synchronize()
        assert bool((whole[0] == -7).all()) and bool((whole[-1] == -7).all()) and bool((whole[:, M:] == -7).all())
        y = whole[1:-1, :M]
        for e in range(last):  # (descending: undefined)
            if what == "beyond" and e == E - 2:
                continue  # (the last offsets are clamped: this one takes the rest)
            cut = torch.arange(e * each, (e + 1) * each, device=DEV)
            cut = cut[fine[cut]]
            assert torch.equal(y[cut], o.product(e, row[cut].long(), dtype)), (what, e)
