"""GPU parity of the int8 rows and products (quantize_i8_rows, pack_i8, qgemm_i8)
against 64-bit references. Quants and scales are compared bit for bit; products
within the float32 epilogue's roundings (beamref.product_tolerance)."""
import numpy as np
import pytest
import torch

import quantized_gemv_argmax_amd as qg
from tests import beamref
from tests.gpu_helpers import DEV, case, to_dev

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = {"f32": 0.0, "f16": 2.0 ** -10, "bf16": 2.0 ** -7}   # one step, relative
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -133}


def check_rows(x, K, what):
    q, scale = qg.quantize_i8_rows(x)
    torch.cuda.synchronize()
    qr, sr = beamref.quantize_rows(x.double().cpu().numpy())
    np.testing.assert_array_equal(scale.cpu().numpy(), sr, err_msg=what)
    np.testing.assert_array_equal(q[:, :K].cpu().numpy(), qr, err_msg=what)
    assert int(q[:, K:].count_nonzero()) == 0, what
    assert q.shape[1] == (K + 63) // 64 * 64


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("N,K", [(1, 1), (3, 7), (1, 64), (5, 65), (2, 1001), (64, 3584), (3, 4097), (1, 18944),
                                 (7, 18945), (2, 40000), (1, 131071), (1030, 64), (600, 3584)])
def test_quantize_rows(N, K, t):
    g = torch.Generator(device=DEV).manual_seed(N * 131 + K)
    case(f"quantize_i8_rows N={N} K={K} {t}")
    x = torch.randn(N, K, generator=g, device=DEV) * torch.exp(2 * torch.randn(N, 1, generator=g, device=DEV))
    check_rows(x.to(TYPES[t]), K, f"{N}x{K} {t}")


@pytest.mark.parametrize("t", list(TYPES))
def test_quantize_strided_rows(t):
    # rows at odd strides and offsets: every alignment of a row's first element
    g = torch.Generator(device=DEV).manual_seed(3)
    base = torch.randn(9, 1103, generator=g, device=DEV).to(TYPES[t])
    for off, K in [(0, 1000), (1, 1001), (3, 512), (5, 65)]:
        case(f"quantize_i8_rows strided offset={off} K={K} {t}")
        check_rows(base[:, off:off + K], K, f"offset {off}")
    # an output with wider rows: bytes beyond the padded K stay as they were
    out = torch.full((9, 1280), 77, dtype=torch.int8, device=DEV)
    qg.quantize_i8_rows(base[:, :1000], out=out)
    assert int((out[:, 1024:] != 77).sum()) == 0 and int(out[:, 1000:1024].count_nonzero()) == 0


def test_quantize_halves_and_extremes():
    # quotients on and next to the halves: d = 1 exactly, then a d that is no power of two
    rows = []
    k = np.arange(-126, 127, dtype=np.float64)
    rows.append(np.concatenate([[127.0], k + 0.5]))
    for d in (1.0, np.float64(np.float32(0.3)), np.float64(np.float32(7.1e-5))):
        near = []
        for h in k + 0.5:
            c = np.float32(h * d)
            near += [c, np.nextafter(c, np.float32(np.inf)), np.nextafter(c, np.float32(-np.inf))]
        rows.append(np.concatenate([[np.float32(127.0 * d)], near]))
    rows += [np.zeros(9), np.array([1e-45, -3e-45, 1.4e-43]), np.array([2e-38, -1e-38, 1e-45, 5e-39]),
             np.array([2.7e-43, 1e-45]), np.array([3.4e38, -1e38, 1e30, 3.0]), np.array([np.nan, 1.0, 2.0]),
             np.array([1.0, np.inf]), np.array([-np.inf, np.nan]), np.array([-0.0, 0.0])]
    for i, r in enumerate(rows):
        case(f"quantize_i8_rows special row {i}")
        x = to_dev(r.astype(np.float32)[None])
        check_rows(x, x.shape[1], f"row {i}")
    h = torch.tensor([[65504.0, -6e-8, 1.0, float("inf")], [6e-8, 1.2e-7, -6e-8, 0.0]], dtype=torch.float16, device=DEV)
    check_rows(h, 4, "fp16")


def operands(M, K, N, seed, full=False):
    rng = np.random.default_rng(seed)
    lo = -128 if full else -127
    wq = rng.integers(lo, 128, (M, K)).astype(np.int8)
    xq = rng.integers(lo, 128, (N, K)).astype(np.int8)
    ws = rng.uniform(1e-4, 2e-3, M).astype(np.float32)
    xs = rng.uniform(1e-3, 5e-2, N).astype(np.float32)
    bias = rng.standard_normal(M).astype(np.float32)
    return wq, xq, ws, xs, bias


def padded(xq, junk=True):
    """Rows of a multiple of 64 bytes; what follows K is arbitrary."""
    N, K = xq.shape
    out = np.full((N, (K + 63) // 64 * 64), 93 if junk else 0, np.int8)
    out[:, :K] = xq
    return out


def check_product(M, K, N, t, bias, seed, full=False):
    wq, xq, ws, xs, b = operands(M, K, N, seed, full)
    case(f"qgemm_i8 M={M} K={K} N={N} {t} bias={bias}")
    wp = qg.pack_i8(to_dev(wq))
    Y = torch.full((N, (M + 3) // 4 * 4 + 4), -7.0, dtype=TYPES[t], device=DEV)
    qg.qgemm_i8(wp, to_dev(ws), to_dev(padded(xq)), to_dev(xs), M, K, bias=to_dev(b) if bias else None, Y=Y)
    torch.cuda.synchronize()
    assert int((Y[:, M:] != -7.0).sum()) == 0  # only M outputs of a row are written
    y = Y[:, :M].double().cpu().numpy()
    yr, p = beamref.product(xq, xs, wq, ws, b if bias else None)
    err, tol = np.abs(y - yr), beamref.product_tolerance(yr, p, EPS[t], TINY[t])
    bad = np.argwhere(~(err <= tol))
    assert not bad.size, f"{len(bad)} off, first {bad[0]}: {y[tuple(bad[0])]} vs {yr[tuple(bad[0])]}"


SHAPES = [(1, 1, 1), (16, 64, 16), (17, 65, 17), (5, 1000, 1), (100, 3, 33), (512, 3584, 1), (3584, 3584, 4),
          (1000, 257, 15), (3584, 18944, 3), (640, 18944, 16), (333, 1001, 31), (4608, 512, 64), (2000, 640, 65),
          (257, 191, 129), (1031, 1024, 255), (700, 2048, 256), (519, 130, 513), (2050, 320, 1000), (384, 18944, 130),
          (520, 9000, 100), (2050, 191, 1537), (2050, 64, 1500), (3300, 200, 4001), (3300, 60, 3900), (3300, 1000, 3900),
          (8200, 3584, 16), (8200, 4096, 31), (9000, 1024, 1), (8195, 1030, 20), (300, 60, 70), (300, 4000, 70), (2600, 500, 300),
          (3600, 4200, 17), (3600, 18944, 32), (3600, 4161, 20), (100, 4161, 20), (6000, 5003, 16), (33, 129, 7), (33, 127, 2)]


@pytest.mark.parametrize("M,K,N", SHAPES)
def test_product(M, K, N):
    for i, (t, bias) in enumerate([("f32", True), ("bf16", False), ("f16", True)]):
        check_product(M, K, N, t, bias, seed=M * 7 + K * 3 + N + i)


def test_product_extreme_sums():
    # the largest K at the largest magnitudes: sums up to 131071 * 128 * 128 = 2^31 - 2^14
    M, K, N = 20, 131071, 3
    wq = np.full((M, K), -128, np.int8)
    xq = np.full((N, K), -128, np.int8)
    xq[1] = 127
    wp = qg.pack_i8(to_dev(wq))
    one = lambda n: torch.ones(n, device=DEV)  # noqa: E731
    case("qgemm_i8 extreme sums")
    y = qg.qgemm_i8(wp, one(M), to_dev(padded(xq)), one(N), M, K)[:, :M].double().cpu().numpy()
    want = xq.astype(np.float64) @ wq.astype(np.float64).T
    np.testing.assert_array_equal(y, want.astype(np.float32).astype(np.float64))


def test_product_nan_scale_stays_in_its_row():
    wq, xq, ws, xs, _ = operands(200, 300, 5, seed=9)
    xs[2] = np.nan
    wp = qg.pack_i8(to_dev(wq))
    case("qgemm_i8 NaN scale")
    y = qg.qgemm_i8(wp, to_dev(ws), to_dev(padded(xq)), to_dev(xs), 200, 300)[:, :200]
    assert bool(y[2].isnan().all()) and not bool(y[[0, 1, 3, 4]].isnan().any())


def test_pack_layout_and_strided_weights():
    M, K = 37, 150
    rng = np.random.default_rng(4)
    base = rng.integers(-128, 128, (M, 163)).astype(np.int8)
    for off in (0, 1, 8):
        w = base[:, off:off + K]
        case(f"pack_i8 strided offset={off}")
        got = qg.pack_i8(to_dev(base)[:, off:off + K]).cpu().numpy().view(np.int8)
        pad = np.zeros((48, 192), np.int8)
        pad[:M, :K] = w
        want = pad.reshape(3, 16, 3, 4, 16).transpose(0, 2, 3, 1, 4).reshape(-1)
        np.testing.assert_array_equal(got, want)


def test_product_same_bits_for_any_number_of_columns():
    # integer sums: a column's outputs do not depend on its neighbours or the form
    M, K = 900, 3584
    wq, xq, ws, xs, b = operands(M, K, 300, seed=21)
    wp, dx, dw, ds, db = qg.pack_i8(to_dev(wq)), to_dev(padded(xq)), to_dev(ws), to_dev(xs), to_dev(b)
    case("qgemm_i8 column independence")
    full = qg.qgemm_i8(wp, dw, dx, ds, M, K, bias=db)[:, :M].clone()
    for n0, n1 in [(0, 1), (3, 8), (0, 16), (10, 42), (5, 69), (0, 128), (7, 264)]:
        part = qg.qgemm_i8(wp, dw, dx[n0:n1], ds[n0:n1].clone(), M, K, bias=db)[:, :M]
        assert torch.equal(part, full[n0:n1]), (n0, n1)


@pytest.mark.parametrize("N", [1, 40, 300])
def test_product_in_graphs_and_on_another_stream(N):
    M, K = 640, 18944
    wq, xq, ws, xs, b = operands(M, K, N, seed=33)
    wp, dx, dw, ds, db = qg.pack_i8(to_dev(wq)), to_dev(padded(xq)), to_dev(ws), to_dev(xs), to_dev(b)
    case(f"qgemm_i8 graph N={N}")
    want = qg.qgemm_i8(wp, dw, dx, ds, M, K, bias=db).clone()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        y = qg.qgemm_i8(wp, dw, dx, ds, M, K, bias=db)
    s.synchronize()
    assert torch.equal(y[:, :M], want[:, :M])
    Ys = [torch.zeros_like(want) for _ in range(2)]
    graphs = []
    for Y in Ys:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            qg.qgemm_i8(wp, dw, dx, ds, M, K, bias=db, Y=Y)
        graphs.append(g)
    for i in range(4):
        for g, Y in zip(graphs, Ys):
            Y.fill_(-1)
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(Ys[0][:, :M], want[:, :M]) and torch.equal(Ys[1][:, :M], want[:, :M]), i
        assert torch.equal(qg.qgemm_i8(wp, dw, dx, ds, M, K, bias=db)[:, :M], want[:, :M])


def test_refusals():
    w = torch.zeros(20, 100, dtype=torch.int8, device=DEV)
    wp, ws = qg.pack_i8(w), torch.ones(20, device=DEV)
    xq, xs = torch.zeros(3, 128, dtype=torch.int8, device=DEV), torch.ones(3, device=DEV)
    ok = dict(M=20, K=100)
    qg.qgemm_i8(wp, ws, xq, xs, **ok)
    for args in [(wp[:-16], ws, xq, xs), (wp, ws[:-1], xq, xs), (wp, ws, xq[:, :64], xs), (wp, ws, xq, xs[:2]),
                 (wp, ws.double(), xq, xs), (wp, ws, xq.float(), xs), (wp.cpu(), ws, xq, xs), (wp, ws.cpu(), xq, xs)]:
        with pytest.raises(ValueError):
            qg.qgemm_i8(*args, **ok)
    with pytest.raises(ValueError):
        qg.qgemm_i8(wp, ws, xq, xs, dtype=torch.float64, **ok)
    with pytest.raises(ValueError):
        qg.qgemm_i8(wp, ws, xq, xs, Y=torch.empty(3, 16, device=DEV), **ok)
    with pytest.raises(qg.QGError):  # rows of Y not a multiple of 4 apart
        qg.qgemm_i8(wp, ws, xq, xs, Y=torch.empty(3, 21, device=DEV), **ok)
    with pytest.raises(ValueError):
        qg.quantize_i8_rows(torch.zeros(3, 4, dtype=torch.float64, device=DEV))
    with pytest.raises(qg.QGError):
        qg.quantize_i8_rows(torch.zeros(0, 4, device=DEV))
    with pytest.raises(ValueError):
        qg.quantize_i8_rows(torch.zeros(3, 4, device=DEV).t())
    with pytest.raises(ValueError):
        qg.pack_i8(torch.zeros(3, 200000, dtype=torch.int8, device=DEV))


FORMS = [("streamed", 100, 300, 5), ("streamed, 32 columns", 500, 300, 20), ("walk", 16500, 1030, 3),
         ("walk, 32 columns", 16500, 1030, 20), ("tiles of 64", 1000, 191, 100), ("tiles of 64, split", 256, 18944, 40),
         ("tiles of 128, three buffers", 1664, 200, 1300), ("tiles of 128, split", 300, 8200, 100),
         ("tiles of 128, two buffers", 4700, 200, 1000), ("tiles of 256", 3300, 200, 4001),
         ("tiles of 256, two for a workgroup", 4300, 200, 4100)]


@pytest.mark.parametrize("form,M,K,N", FORMS)
def test_product_and_bias_are_rounded_once(form, M, K, N):
    """Every form bit for bit: the sum to float32, the scales' product to float32, product
    and bias in one rounding, one more to a 16-bit output."""
    wq, xq, ws, xs, _ = operands(M, K, N, seed=M + K + N)
    rng = np.random.default_rng(M)
    b = (rng.standard_normal(M) * 40 * np.sqrt(K) * ws * xs.mean()).astype(np.float32)  # as large as the products
    acc = (torch.from_numpy(xq).double() @ torch.from_numpy(wq).double().t()).numpy().astype(np.float32)
    scale = xs[:, None] * ws[None]
    want = torch.from_numpy(beamref.fused32(acc, scale, np.broadcast_to(b, scale.shape)))
    assert bool((want != torch.from_numpy(acc * scale + b)).any())  # two roundings are told apart
    wp, dx, dw, ds, db = qg.pack_i8(to_dev(wq)), to_dev(padded(xq)), to_dev(ws), to_dev(xs), to_dev(b)
    for t, dtype in TYPES.items():
        case(f"qgemm_i8 {form} M={M} K={K} N={N} {t} rounded once")
        y = qg.qgemm_i8(wp, dw, dx, ds, M, K, bias=db, dtype=dtype)[:, :M].cpu()
        assert torch.equal(y, want.to(dtype)), (form, t, int((y != want.to(dtype)).sum()))
