"""The gated rows of quantize_f8_rows over the whole range of their gates, against 64 bits: gates whose
exponential passes float32, factors below the normal floats, infinities and NaN."""
import numpy as np
import pytest
import torch

import quantized_gemv_argmax_amd as qg
from tests import f8ref
from tests.gpu_helpers import DEV, case

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
INF, NAN = float("inf"), float("nan")


def check(x, what):
    """Rows of whole blocks of 128 against float64. The gate's factor: two units in the last place of the
    hardware's exponential and reciprocal, a sum and three products, together below 2^-20; below the normal floats
    a step of 2^-149. Its product with u: half a unit, or such a step. The scale: half a unit, or such a step.
    A value: half a step of its octave, and where the scale is below the normal floats what it is clamped by."""
    K = x.shape[1] // 2
    q, s = qg.quantize_f8_rows(x, gated=True)
    torch.cuda.synchronize()
    v = x.double().cpu().numpy()
    with np.errstate(invalid="ignore", over="ignore"):
        u, h = np.abs(v[:, K:]), f8ref.silu_gate(v[:, :K], v[:, K:])
    codes, scale = q.view(torch.uint8).cpu().numpy(), s.double().cpu().numpy()
    with np.errstate(invalid="ignore"):
        off = np.abs(h) * 2.0 ** -20 + (u + 1) * 2.0 ** -149
    for b in range(K // 128):
        cut = slice(128 * b, 128 * b + 128)
        for n in range(x.shape[0]):
            hb, ob, d, c, where = h[n, cut], off[n, cut], scale[n, b], codes[n, cut], f"{what}, row {n}, block {b}"
            if not np.isfinite(hb).all():
                assert np.isnan(d) and not c.any(), where
                continue
            top = np.abs(hb).max()
            assert abs(d - top / 448) <= (ob.max() + top * 2.0 ** -24) / 448 + 2.0 ** -150, (where, d, top / 448)
            if d == 0:
                assert not c.any(), where
                continue
            octave = 2.0 ** np.floor(np.log2(np.maximum(np.abs(hb) / d, 2.0 ** -6)))
            tol = octave / 16 * (1 + 2.0 ** -18) * d + ob + (448 * 2.0 ** -150 if d < 2.0 ** -126 else 0)
            assert (np.abs(f8ref.VALUES[c] * d - hb) <= tol).all(), where


def blocks(gates, ups, t):
    """One row, a block of 128 for each pair."""
    g = torch.tensor([[a for a in gates for _ in ups]], dtype=torch.float64).repeat_interleave(128, 1)
    u = torch.tensor([[b for _ in gates for b in ups]], dtype=torch.float64).repeat_interleave(128, 1)
    return torch.cat([g, u], 1).to(DEV).to(TYPES[t])


@pytest.mark.parametrize("t", list(TYPES))
def test_far_gates(t):
    # about -87.34 the exponential passes 2^126, at -88.73 float32; below -103.98 it is less than the smallest float
    gates = [-60, -64, -86.9, -87, -87.3, -87.34, -87.5, -88, -88.6, -88.72, -88.73, -89, -92, -95, -100, -103, -104, -105, -120, -133,
             -140, -200, -1000, 60, 86.9, 87, 87.5, 88.5, 90, 130, 1000, 0.0, -0.0]
    ups = [1e4, -1.0, 3e-5, 0.0] + ([1e20, -3e30] if t != "f16" else [65504.0])
    case(f"quantize_f8_rows far gates {t}")
    check(blocks(gates, ups, t), f"far gates {t}")
    if t != "f16":
        check(blocks([-1e30, -3.3e38, 1e30, 3.3e38], [1.0, 1e-30, 0.0], t), f"farthest gates {t}")


@pytest.mark.parametrize("t", list(TYPES))
def test_far_gates_among_others(t):
    """A far gate in a lane, among common ones in the same lane and in others."""
    g = torch.Generator(device=DEV).manual_seed(5)
    x = torch.randn(12, 2 * 1024, generator=g, device=DEV) * 4
    for n in range(1, 12):
        x[n, n * 83 % 1024] = [-88, -87.5, -95, 90, -120, 88, -87, -200, -89, 300, -104][n - 1]
        x[n, 1024 + n * 83 % 1024] = 1e4
    x[11, :1024] = torch.linspace(-130, 130, 1024, device=DEV)
    case(f"quantize_f8_rows far gates among others {t}")
    check(x.to(TYPES[t]), f"mixed {t}")


@pytest.mark.parametrize("t", list(TYPES))
def test_gates_and_factors_that_are_not_finite(t):
    rows = []
    for gate, up in [(INF, 1.0), (-INF, 1.0), (NAN, 1.0), (1.0, INF), (1.0, -INF), (1.0, NAN), (INF, 0.0), (-INF, 0.0), (-1000.0, INF)]:
        r = torch.ones(1, 2 * 384)
        r[0, 130], r[0, 384 + 130] = gate, up
        rows.append(r)
    x = torch.cat(rows).to(DEV).to(TYPES[t])
    case(f"quantize_f8_rows gates that are not finite {t}")
    check(x, f"not finite {t}")
    _, s = qg.quantize_f8_rows(x, gated=True)
    assert torch.isnan(s[:, :3]).tolist() == [[False, True, False]] * len(rows)
