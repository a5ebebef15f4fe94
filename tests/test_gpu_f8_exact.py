"""Every form of the e4m3 products bit for bit, on operands whose sums are exact: a product that is left
out, taken twice or met with another block's scale shows. The large tiles are walked past a workgroup's
first one, with numbers of blocks from the least that they take on, even and odd, and tile rows that
end inside the matrix."""
import pytest
import torch

import quantized_gemv_argmax_amd as qg
from tests import f8ref
from tests.f8exact import DEV, F8, Operands, units, up
from tests.gpu_helpers import case, to_dev

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.fixture(autouse=True)
def give_back_memory():
    yield
    torch.cuda.empty_cache()


def check_dense(M, K, N, dtype, bias, seed):
    case(f"qgemm_f8 exact M={M} K={K} N={N} {dtype} bias={bias}")
    o = Operands(1, M, K, N, seed, bias)
    w = qg.pack_f8(o.w[0])
    Y = torch.full((N, up(M, 4) + 4), -7.0, dtype=dtype, device=DEV)
    qg.qgemm_f8(w, o.ws[0], o.xq, o.xs, M, K, bias=o.bias[0] if bias else None, Y=Y)
    assert torch.equal(Y[:, :M], o.product(0, slice(None), dtype))
    assert bool((Y[:, M:] == -7.0).all())
    again = qg.qgemm_f8(w, o.ws[0], o.xq, o.xs, M, K, bias=o.bias[0] if bias else None, dtype=dtype)
    assert torch.equal(again[:, :M], Y[:, :M])


# few rows; tiles of 64, whole and split; 128 x 64; tiles of 128, whole and split; tiles of 128 below four blocks
@pytest.mark.parametrize("M,K,N", [(333, 1001, 3), (8192, 300, 16), (517, 1001, 77), (300, 7400, 40), (66000, 300, 33),
                                   (2050, 700, 1000), (260, 9000, 100), (5300, 384, 5300)])
def test_product(M, K, N):
    for i, dtype in enumerate((F32, BF16, F16)):
        check_dense(M, K, N, dtype, i != 1, seed=M + K + N + i)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("M,K,N", [(5300, 385, 5300), (5300, 512, 5300), (5376, 512, 9000), (5300, 640, 5300), (5300, 640, 9001),
                                   (5300, 700, 5376), (5300, 1100, 5300)])
def test_product_walks_tiles_of_256(M, K, N, dtype):
    whole, half = -(-M // 256) * -(-N // 256), -(-M // 256) * -(-N // 128)
    rounds = [-(-t // units()) for t in (whole, half)]
    assert whole > units() and rounds[0] * 9 <= rounds[1] * 5 and K > 384  # (what takes these tiles)
    check_dense(M, K, N, dtype, dtype == F16, seed=M + K + N)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("M,K,N", [(4700, 385, 4200), (4700, 512, 4200), (4608, 512, 4224), (4700, 640, 4200), (4700, 700, 4200)])
def test_product_walks_tiles_of_256x128(M, K, N, dtype):
    whole, half = -(-M // 256) * -(-N // 256), -(-M // 256) * -(-N // 128)
    rounds = [-(-t // units()) for t in (whole, half)]
    assert half > units() and rounds[0] * 9 > rounds[1] * 5 and K > 384
    check_dense(M, K, N, dtype, dtype == F16, seed=M + K + N)


def check_grouped(M, K, counts, dtype, bias, gather, seed):
    case(f"qgemm_f8_grouped exact M={M} K={K} rows={sum(counts)} of {len(counts)} {dtype} bias={bias} gather={gather}")
    E, lead, tail = len(counts), 3, 5
    R = lead + sum(counts) + tail
    X = R // 2 + 1 if gather else R
    o = Operands(E, M, K, X, seed, bias)
    g = torch.Generator(device=DEV).manual_seed(seed + 1)
    row = torch.randint(0, X, (R,), generator=g, device=DEV, dtype=torch.int32) if gather else None
    at = [lead]
    for c in counts:
        at.append(at[-1] + c)
    offsets = torch.tensor(at, dtype=torch.int32, device=DEV)
    Y = torch.full((R, up(M, 4) + 4), -7.0, dtype=dtype, device=DEV)
    args = (qg.pack_f8(o.w), o.ws, o.xq, o.xs, M, K, offsets)
    qg.qgemm_f8_grouped(*args, row=row, bias=o.bias, Y=Y)
    for e in range(E):
        cut = slice(at[e], at[e + 1])
        rows = cut if row is None else row[cut].long()
        assert torch.equal(Y[cut, :M], o.product(e, rows, dtype)), e
    assert bool((Y[:, M:] == -7.0).all()) and bool((Y[:lead] == -7.0).all()) and bool((Y[at[-1]:] == -7.0).all())
    again = qg.qgemm_f8_grouped(*args, row=row, bias=o.bias, dtype=dtype)
    assert torch.equal(again[lead:at[-1], :M], Y[lead:at[-1], :M])


# streamed; tiles of 64; of 128 x 64; of 128
@pytest.mark.parametrize("M,K,counts", [(130, 700, [3, 0, 4, 1]), (400, 300, [1, 2, 0, 3, 1, 2] * 10), (300, 700, [40, 0, 33, 70]),
                                        (600, 384, [100] * 60), (1100, 384, [700] * 20)])
def test_grouped(M, K, counts):
    for i, dtype in enumerate((F32, BF16, F16)):
        check_grouped(M, K, counts, dtype, i != 1, i != 2, seed=M + K + i)


EVEN = [700] * 20
UNEVEN = [513, 1, 900, 0, 1300, 255, 256, 257, 1024, 700] * 2 + [2000, 1, 0, 600]
GATHERS = [(BF16, False), (F16, True), (BF16, True)]


@pytest.mark.parametrize("dtype,gather", GATHERS)
@pytest.mark.parametrize("M,K,counts", [(1100, 385, EVEN), (1100, 512, EVEN), (1100, 512, UNEVEN), (1280, 640, UNEVEN), (1100, 700, UNEVEN),
                                        (1100, 1100, EVEN)])
def test_grouped_walks_tiles_of_256(M, K, counts, dtype, gather):
    assert sum(counts) >= 512 * len(counts) and K > 384  # (what takes these tiles)
    assert sum(-(-c // 256) for c in counts) * -(-M // 256) > units()
    check_grouped(M, K, counts, dtype, gather, gather, seed=M + K)


@pytest.mark.parametrize("dtype,gather", GATHERS)
@pytest.mark.parametrize("M,K,counts", [(600, 385, [100] * 120), (600, 512, [100] * 120), (768, 512, [300, 70, 129, 0, 1] * 30),
                                        (600, 640, [300, 70, 129, 0, 1] * 40), (1000, 1100, [257, 0, 1, 400] * 20)])
def test_grouped_walks_tiles_of_256x128(M, K, counts, dtype, gather):
    mean = sum(counts) / len(counts)
    assert 64 < mean < 500 and K > 384
    assert sum(-(-c // 128) for c in counts) * -(-M // 256) > units()
    check_grouped(M, K, counts, dtype, gather, gather, seed=M + K)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("first", [0, 7, 60, 63, 100, 126])
def test_products_down_to_2_13_of_the_largest_count(first, dtype):
    """Two products of 2^14 and -2^14 and one of 2^(14 - g), anywhere in the block: what is
    left is that one, of the 8-bit matrix cores down to g = 13; below, it may be lost."""
    case(f"qgemm_f8 single products beside {first} {dtype}")
    at = [j for j in range(128) if j not in (first, first + 1)]
    x = torch.zeros(len(at), 128, dtype=torch.float64)
    x[:, first] = x[:, first + 1] = 128.0
    for n, j in enumerate(at):
        x[n, j] = 128.0
    w = (128.0 * 2.0 ** -torch.arange(17, dtype=torch.float64))[:, None].repeat(1, 128)
    w[:, first], w[:, first + 1] = 128.0, -128.0
    want = (2.0 ** (14 - torch.arange(17, dtype=torch.float64)))[None].repeat(len(at), 1)
    f8 = [to_dev(f8ref.encode(v.numpy())).view(F8) for v in (x, w)]
    ones = torch.ones(len(at), 4, device=DEV)
    y = qg.qgemm_f8(qg.pack_f8(f8[1]), ones[:1, :1].contiguous(), f8[0], ones, 17, 128, dtype=dtype)[:, :17].double().cpu()
    assert torch.equal(y[:, :14], want[:, :14])
    assert bool(((y[:, 14:] - want[:, 14:]).abs() <= want[:, 14:]).all())
    y = qg.qgemm_f8(qg.pack_f8(f8[1]), ones[:1, :1].contiguous(), f8[0], ones, 17, 128)[:, :17].double().cpu()
    assert torch.equal(y, want)  # float32 outputs lose none


@pytest.mark.parametrize("M,K,N", [(64, 128, 64), (517, 1001, 77), (2050, 700, 1000), (4700, 520, 4200)])
def test_random_bytes(M, K, N):
    """Values of the whole range, so that most of a block's products lie far below its largest:
    within the bound of the 8-bit matrix cores that f8ref.product derives, and the float32 outputs' own."""
    case(f"qgemm_f8 random bytes M={M} K={K} N={N}")
    g = torch.Generator(device=DEV).manual_seed(M + N)
    nb = -(-K // 128)

    def draw(r):
        c = torch.randint(0, 256, (r, K), generator=g, device=DEV, dtype=torch.uint8)
        return torch.where((c & 0x7F) == 0x7F, torch.zeros_like(c), c)

    wc, xc = draw(M), draw(N)
    xq = torch.zeros(N, nb * 128, dtype=torch.uint8, device=DEV)
    xq[:, :K] = xc
    ws = torch.rand(-(-M // 128), nb, generator=g, device=DEV) * 1e-4 + 1e-5
    xs = torch.rand(N, up(nb, 4), generator=g, device=DEV) * 1e-2 + 1e-3
    wv = wc.view(F8).double() * ws.double().repeat_interleave(128, 0)[:M].repeat_interleave(128, 1)[:, :K]
    xv = xc.view(F8).double() * xs.double().repeat_interleave(128, 1)[:, :K]
    ref = torch.mm(xv, wv.t().contiguous())
    mag = torch.mm(xv.abs(), wv.abs().t().contiguous())
    for dtype, half, tiny in ((F32, 2.0 ** -24, 2.0 ** -149), (BF16, 2.0 ** -8, 2.0 ** -133), (F16, 2.0 ** -11, 2.0 ** -25)):
        y = qg.qgemm_f8(qg.pack_f8(wc.view(F8)), ws, xq.view(F8), xs, M, K, dtype=dtype)[:, :M].double()
        tol = mag * (128 + 3 + nb + 16) * 2.0 ** -23 + (0 if dtype == F32 else mag * 7 * 2.0 ** -13)
        tol = tol + (ref.abs() + tol) * half + tiny
        assert bool(((y - ref).abs() <= tol).all()), dtype
