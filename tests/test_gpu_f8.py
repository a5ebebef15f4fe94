"""GPU parity of the block-scaled e4m3 rows and products (quantize_f8_rows, pack_f8,
qgemm_f8, qgemm_f8_grouped) against 64-bit references. Codes and scales are compared bit
for bit; products within the bounds that f8ref.product derives."""
import numpy as np
import pytest
import torch

import quantized_gemv_argmax_amd as qg
from tests import f8ref
from tests.gpu_helpers import DEV, case, to_dev

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}  # half a step, relative
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -133}
F8 = torch.float8_e4m3fn


def f8(codes):
    return to_dev(codes).view(F8)


def check_rows(x, what, gated=False):
    K = x.shape[1] // (2 if gated else 1)
    q, scale = qg.quantize_f8_rows(x, gated=gated)
    torch.cuda.synchronize()
    nb = (K + 127) // 128
    assert q.dtype == F8 and q.shape == (x.shape[0], nb * 128) and scale.shape == (x.shape[0], (nb + 3) // 4 * 4)
    qc, sc = q.view(torch.uint8).cpu().numpy(), scale.cpu().numpy()
    assert not qc[:, K:].any() and not sc[:, nb:].any(), what
    h = x.double().cpu().numpy()
    if not gated:
        want, ws = f8ref.quantize_rows(h)
        np.testing.assert_array_equal(sc[:, :nb], ws, err_msg=what)
        np.testing.assert_array_equal(qc[:, :K], want, err_msg=what)
        return
    # float32: the exponential (2^-21 with its argument's rounding), a sum, a quotient, a product
    h = f8ref.silu_gate(h[:, :K], h[:, K:])
    with np.errstate(invalid="ignore"):
        e = np.abs(h) * 2.0 ** -20
    for b in range(nb):
        cut = slice(128 * b, min(K, 128 * b + 128))
        top = np.abs(h[:, cut]).max(1)
        s = sc[:, b].astype(np.float64)
        assert (np.abs(s - top / 448) <= top / 448 * 2.0 ** -20 + 2.0 ** -149).all(), what
        v = f8ref.VALUES[qc[:, cut]] * s[:, None]
        # half a step of the value's octave (a step is at most 2^-3 of the value; 2^-9 at least)
        step = np.maximum(2.0 ** np.floor(np.log2(np.maximum(np.abs(h[:, cut]) / np.maximum(s, 1e-300)[:, None], 2.0 ** -6))), 2.0 ** -6) / 8
        assert (np.abs(v - h[:, cut]) <= (step / 2 * (1 + 2.0 ** -18)) * s[:, None] + e[:, cut]).all(), what


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("N,K", [(1, 1), (3, 7), (1, 128), (5, 129), (2, 1001), (64, 3584), (3, 513), (1, 18944), (7, 18945),
                                 (1, 131072), (4097, 64), (700, 3584)])
def test_quantize_rows(N, K, t):
    g = torch.Generator(device=DEV).manual_seed(N * 131 + K)
    case(f"quantize_f8_rows N={N} K={K} {t}")
    x = torch.randn(N, K, generator=g, device=DEV) * torch.exp(2 * torch.randn(N, 1, generator=g, device=DEV))
    check_rows(x.to(TYPES[t]), f"{N}x{K} {t}")


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("N,K", [(1, 1), (3, 7), (5, 129), (2, 1001), (64, 768), (1, 18944), (700, 1536)])
def test_quantize_gated_rows(N, K, t):
    g = torch.Generator(device=DEV).manual_seed(N * 17 + K)
    case(f"quantize_f8_rows gated N={N} K={K} {t}")
    x = torch.randn(N, 2 * K, generator=g, device=DEV) * 4
    check_rows(x.to(TYPES[t]), f"{N}x{K} {t}", gated=True)


@pytest.mark.parametrize("t", list(TYPES))
def test_quantize_strided_rows(t):
    # rows at odd strides and offsets: every alignment of a row's first element
    g = torch.Generator(device=DEV).manual_seed(3)
    base = torch.randn(9, 1103, generator=g, device=DEV).to(TYPES[t])
    for off, K in [(0, 1000), (1, 1001), (3, 512), (5, 65)]:
        case(f"quantize_f8_rows strided offset={off} K={K} {t}")
        check_rows(base[:, off:off + K], f"offset {off}")
        check_rows(base[:, off:off + K // 2 * 2], f"gated, offset {off}", gated=True)


def test_quantize_leaves_what_lies_beyond():
    x = torch.randn(9, 1000, device=DEV)
    out = torch.full((9, 1280), 77, dtype=torch.uint8, device=DEV).view(F8)
    scale = torch.full((9, 12), 5.0, device=DEV)
    case("quantize_f8_rows into wider rows, 4 of 9")
    qg.quantize_f8_rows(x, count=torch.tensor([4], dtype=torch.int32, device=DEV), out=out, scale=scale)
    torch.cuda.synchronize()
    raw = out.view(torch.uint8)
    assert int((raw[:, 1024:] != 77).sum()) == 0 and int((raw[4:] != 77).sum()) == 0 and int(raw[:4, 1000:1024].count_nonzero()) == 0
    assert int((scale[:, 8:] != 5).sum()) == 0 and int((scale[4:] != 5).sum()) == 0
    want, ws = f8ref.quantize_rows(x[:4].double().cpu().numpy())
    np.testing.assert_array_equal(raw[:4, :1000].cpu().numpy(), want)
    np.testing.assert_array_equal(scale[:4, :8].cpu().numpy(), ws)
    for n in (0, -3, 100):  # none, and more than there are
        qg.quantize_f8_rows(x, count=torch.tensor([n], dtype=torch.int32, device=DEV), out=out, scale=scale)
        assert int((raw[8, :1000] != 77).any()) == (n > 0)


def test_quantize_borders_and_extremes():
    # quotients on and next to every border between two values, for scales that are powers of two and others
    rows = []
    for d in (1.0, 2.0 ** -7, np.float64(np.float32(0.3)), np.float64(np.float32(7.1e-5))):
        vals = [np.float32(448.0 * d)]
        for h in f8ref.BORDERS:
            c = np.float32(h * d)
            vals += [c, -c, np.nextafter(c, np.float32(np.inf)), np.nextafter(c, np.float32(-np.inf))]
        vals = np.array(vals, np.float32)
        blocks = [np.concatenate([vals[:1], vals[1 + 127 * i:1 + 127 * (i + 1)]]) for i in range(-(-(len(vals) - 1) // 127))]
        rows.append(np.concatenate(blocks))  # 448 d in every block: the scale is d
    rows += [np.zeros(9), np.array([1e-45, -3e-45, 1.4e-43]), np.array([2e-38, -1e-38, 1e-45, 5e-39]), np.array([6e-43, 1e-45]),
             np.array([3.4e38, -1e38, 1e30, 3.0]), np.array([np.nan, 1.0, 2.0]), np.array([1.0, np.inf]),
             np.array([-np.inf, np.nan]), np.array([-0.0, 0.0]), np.array([-448.0, 464.0, 447.0])]
    for i, r in enumerate(rows):
        case(f"quantize_f8_rows special row {i}")
        check_rows(to_dev(np.asarray(r, np.float32)[None]), f"row {i}")
    case("quantize_f8_rows: a NaN stays in its block")
    x = torch.ones(1, 400, device=DEV)
    x[0, 130] = float("nan")
    q, s = qg.quantize_f8_rows(x)
    assert torch.isnan(s[0]).tolist() == [False, True, False, False] and int(q.view(torch.uint8)[0, 128:256].count_nonzero()) == 0


def codes(shape, rng, spread=110):
    return f8ref.encode(rng.standard_normal(shape) * spread)


def padded(c, junk=None):
    """Rows of whole blocks, zeros beyond K."""
    out = np.zeros((c.shape[0], (c.shape[1] + 127) // 128 * 128), np.uint8)
    out[:, :c.shape[1]] = c
    return out


def scales(N, K, rng):
    nb = (K + 127) // 128
    s = np.full((N, (nb + 3) // 4 * 4), np.nan, np.float32)  # what lies beyond the blocks may be anything
    s[:, :nb] = rng.uniform(1e-3, 5e-3, (N, nb))
    return s


def weight_scales(M, K, rng):
    return rng.uniform(1e-4, 3e-4, ((M + 127) // 128, (K + 127) // 128)).astype(np.float32)


def compare(y, ref, t, wide):
    """wide: whether the 8-bit matrix cores may have added (16-bit outputs of more than a few rows)."""
    yr, e32, e8 = ref
    tol = e32 + (e8 if wide and t != "f32" else 0)
    tol = tol + (np.abs(yr) + tol) * HALF[t] + TINY[t]
    bad = np.argwhere(~(np.abs(y - yr) <= tol))
    assert not bad.size, f"{len(bad)} off, first {bad[0]}: {y[tuple(bad[0])]} vs {yr[tuple(bad[0])]} within {tol[tuple(bad[0])]}"


def check_product(M, K, N, t, bias, seed):
    rng = np.random.default_rng(seed)
    wc, xc, ws, xs = codes((M, K), rng), codes((N, K), rng, 150), weight_scales(M, K, rng), scales(N, K, rng)
    b = rng.standard_normal(M).astype(np.float32) if bias else None
    case(f"qgemm_f8 M={M} K={K} N={N} {t} bias={bias}")
    wp = qg.pack_f8(f8(wc))
    Y = torch.full((N, (M + 3) // 4 * 4 + 4), -7.0, dtype=TYPES[t], device=DEV)
    qg.qgemm_f8(wp, to_dev(ws), f8(padded(xc)), to_dev(xs), M, K, bias=to_dev(b) if bias else None, Y=Y)
    torch.cuda.synchronize()
    assert int((Y[:, M:] != -7.0).sum()) == 0  # only M outputs of a row are written
    compare(Y[:, :M].double().cpu().numpy(), f8ref.product(xc, xs, wc, ws, b), t, N > 1)


SHAPES = [(1, 1, 1), (16, 128, 16), (17, 129, 17), (5, 1000, 1), (100, 3, 33), (512, 3584, 1), (1000, 257, 15), (640, 18944, 16),
          (333, 1001, 31), (2000, 640, 65), (257, 191, 129), (1031, 1024, 255), (700, 2048, 256), (519, 130, 513),
          (2050, 320, 1000), (384, 18944, 130), (520, 9000, 100), (2050, 191, 1537), (3300, 200, 4001), (3300, 1000, 3900),
          (8200, 3584, 16), (8195, 1030, 20), (300, 4000, 70), (3600, 4161, 20), (33, 129, 7), (130, 18944, 64), (64, 18944, 40), (9000, 600, 5), (9000, 600, 40), (70000, 300, 50), (4700, 520, 4200), (5000, 300, 4300), (3000, 1030, 1500), (4000, 520, 900), (4650, 1100, 4250), (6000, 1700, 3000)]


@pytest.mark.parametrize("M,K,N", SHAPES)
def test_product(M, K, N):
    for i, (t, bias) in enumerate([("f32", True), ("bf16", False), ("f16", True)]):
        check_product(M, K, N, t, bias, seed=M * 7 + K * 3 + N + i)


def ragged(counts, rng, lead=0):
    offsets = np.concatenate([[lead], lead + np.cumsum(counts)]).astype(np.int32)
    return offsets


def check_grouped(M, K, counts, t, bias, gather, seed, lead=0, tail=0, X=None):
    rng = np.random.default_rng(seed)
    E, offsets = len(counts), ragged(counts, rng, lead)
    R = int(offsets[-1]) + tail
    X = X or (max(1, R // 2) if gather else R)
    wc, ws = codes((E, M, K), rng), np.stack([weight_scales(M, K, rng) for _ in range(E)])
    xc, xs = codes((X, K), rng, 150), scales(X, K, rng)
    row = rng.integers(0, X, R).astype(np.int32) if gather else None
    b = rng.standard_normal((E, M)).astype(np.float32) if bias else None
    case(f"qgemm_f8_grouped E={E} M={M} K={K} R={R} {t} bias={bias} gather={gather}")
    wp = qg.pack_f8(f8(wc))
    Y = torch.full((R, (M + 3) // 4 * 4 + 4), -7.0, dtype=TYPES[t], device=DEV)
    qg.qgemm_f8_grouped(wp, to_dev(ws), f8(padded(xc)), to_dev(xs), M, K, to_dev(offsets), row=None if row is None else to_dev(row),
                        bias=to_dev(b) if bias else None, Y=Y)
    torch.cuda.synchronize()
    assert int((Y[:, M:] != -7.0).sum()) == 0 and int((Y[:lead] != -7.0).sum()) == 0 and int((Y[int(offsets[-1]):] != -7.0).sum()) == 0
    y = Y[:, :M].double().cpu().numpy()
    for e in range(E):
        a, z = offsets[e], offsets[e + 1]
        of = np.arange(a, z) if row is None else row[a:z]
        if z > a:
            compare(y[a:z], f8ref.product(xc[of], xs[of], wc[e], ws[e], None if b is None else b[e]), t, True)


GROUPS = [(64, 128, [1]), (17, 129, [3, 0, 40]), (517, 1001, [0, 2, 1, 0, 5, 33, 0, 1] * 4), (256, 384, [0, 0, 0, 0]),
          (300, 700, [70, 1, 0, 64, 65, 200]), (140, 260, [130, 300, 128, 0, 1, 500]), (1536, 2048, [8, 30, 17, 0, 16, 1]),
          (384, 256, [260, 700, 0, 255, 257, 513]), (2100, 640, [300, 70, 129] * 8), (1000, 1100, [257, 0, 1, 400] * 10 + [900]), (600, 512, [100] * 60), (700, 700, [900, 1, 513, 700]), (1100, 520, [700] * 13), (2300, 1537, [200] * 20),
          (96, 640, [1] * 130), (100, 130, [0] * 70 + [45] + [0] * 60 + [2]), (260, 300, [900])]


@pytest.mark.parametrize("M,K,counts", GROUPS)
def test_grouped(M, K, counts):
    for i, (t, bias, gather) in enumerate([("f32", True, True), ("bf16", False, False), ("f16", True, True)]):
        check_grouped(M, K, counts, t, bias, gather, seed=M * 5 + K + len(counts) + i, lead=0 if i == 0 else 3, tail=0 if i == 1 else 5)


@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_grouped_by_many_experts(t):
    counts = np.random.default_rng(4).integers(0, 3, 1024)
    check_grouped(40, 200, counts.tolist(), t, False, True, seed=5)
    counts = np.zeros(1024, np.int64)
    counts[[0, 63, 64, 700, 1023]] = [400, 300, 10, 129, 350]
    check_grouped(40, 200, counts.tolist(), t, False, True, seed=6)


def test_grouped_with_few_source_rows():
    # every row of Y comes from one of two rows of xq
    check_grouped(130, 300, [50, 0, 90], "bf16", False, True, seed=7, X=2)
    check_grouped(130, 300, [5, 0, 9], "f32", False, True, seed=7, X=2)


def test_grouped_indices_out_of_range_stay_in_bounds():
    # what such rows get is undefined; the others, and what lies around, are not touched
    rng = np.random.default_rng(11)
    M, K, E, R, X = 96, 256, 4, 160, 20
    wc, ws = codes((E, M, K), rng), np.stack([weight_scales(M, K, rng) for _ in range(E)])
    xc, xs = codes((X, K), rng, 150), scales(X, K, rng)
    row = rng.integers(0, X, R).astype(np.int32)
    row[7], row[100] = -5, X + 1000
    for offsets in ([0, 40, 90, 150, R], [0, 40, 90, R + 500, 1 << 30], [-9, 40, 90, 60, R]):
        case(f"qgemm_f8_grouped offsets {offsets}")
        whole = torch.full((R + 2, 100), -7.0, device=DEV)
        qg.qgemm_f8_grouped(qg.pack_f8(f8(wc)), to_dev(ws), f8(padded(xc)), to_dev(xs), M, K, to_dev(np.array(offsets, np.int32)),
                            row=to_dev(row), Y=whole[1:-1])
        torch.cuda.synchronize()
        assert int((whole[0] != -7).sum()) == 0 and int((whole[-1] != -7).sum()) == 0 and int((whole[:, M:] != -7).sum()) == 0
        ok = np.setdiff1d(np.arange(40), [7])
        y = whole[1:-1, :M].double().cpu().numpy()
        compare(y[ok], f8ref.product(xc[row[ok]], xs[row[ok]], wc[0], ws[0]), "f32", True)


def test_pack_takes_strided_weights():
    rng = np.random.default_rng(2)
    base = codes((3, 50, 400), rng)
    d = f8(base)
    for cut in (d[:, 1:38, 3:260], d[1:2, :, :129], d[:, :1, 5:6]):
        case(f"pack_f8 {tuple(cut.shape)} strides {cut.stride()}")
        whole = cut.view(torch.uint8).contiguous().view(F8)
        assert torch.equal(qg.pack_f8(cut), qg.pack_f8(whole))
    # the layout: (t, i, b, h, g, j, l) is row 32 t + 8 j + 4 i + l, k = 128 b + 64 h + 16 g ..
    w = base[0, :37, :260]
    want = np.zeros((64, 384), np.uint8)
    want[:37, :260] = w
    want = want.reshape(2, 4, 2, 4, 3, 2, 4, 16).transpose(0, 2, 4, 5, 6, 1, 3, 7).reshape(-1)
    np.testing.assert_array_equal(qg.pack_f8(f8(w)).cpu().numpy(), want)


def test_nan_scales_stay_in_their_rows():
    rng = np.random.default_rng(9)
    M, K, N = 200, 300, 70
    wc, xc, ws, xs = codes((M, K), rng), codes((N, K), rng), weight_scales(M, K, rng), scales(N, K, rng)
    xs[2, 1] = np.nan
    for n in (5, N):
        y = qg.qgemm_f8(qg.pack_f8(f8(wc)), to_dev(ws), f8(padded(xc[:n])), to_dev(xs[:n]), M, K, dtype=torch.bfloat16)[:, :M]
        nan = torch.isnan(y).cpu().numpy()
        assert nan[2].all() and not np.delete(nan, 2, 0).any()
