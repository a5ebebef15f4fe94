"""The e4m3 and expert operators on rows far apart, whose byte offsets pass 2^31 and 2^32, and on
two streams at once: the same bits as on compact rows (which are tested against 64-bit references) and as
one after the other."""
import pytest
import torch

import quantized_gemv_argmax_amd as qg
from tests.gpu_helpers import DEV, case

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn


@pytest.fixture(autouse=True)
def give_back_memory():
    yield
    torch.cuda.empty_cache()


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def apart(t, ld):
    """t with rows ld elements apart (what lies between them is not set)."""
    whole = torch.empty(((t.shape[0] - 1) * ld + t.shape[1],), dtype=t.dtype, device=DEV)
    far = whole.as_strided(t.shape, (ld, 1))
    far.copy_(t)
    return far


def bits(t):
    return t.contiguous().view(torch.uint8)


def operands(E, M, K, X, g):
    w = (torch.randn(E, M, K, generator=g, device=DEV) * 100).clamp(-448, 448).to(F8)
    ws = torch.rand(E, -(-M // 128), -(-K // 128), generator=g, device=DEV) + 0.5
    xq, xs = qg.quantize_f8_rows(torch.randn(X, K, generator=g, device=DEV))
    return qg.pack_f8(w), ws, xq, xs


@pytest.mark.parametrize("gated", [False, True])
def test_quantize_far_rows(gated):
    case(f"quantize_f8_rows rows 2^26 apart gated={gated}")
    x = torch.randn(40, 600, generator=gen(1), device=DEV).bfloat16()
    q, s = qg.quantize_f8_rows(x, gated=gated)
    far_q, far_s = apart(torch.zeros_like(q), 1 << 27), apart(torch.zeros_like(s), 1 << 25)
    qg.quantize_f8_rows(apart(x, 1 << 26), gated=gated, out=far_q, scale=far_s)
    assert torch.equal(bits(far_q), bits(q)) and torch.equal(far_s, s)


# few columns, tiles of 64, tiles of 128, large tiles (float32: without turns)
@pytest.mark.parametrize("M,K,N", [(130, 300, 14), (260, 520, 1100), (1028, 700, 1100), (2100, 700, 2304), (4164, 640, 2304)])
def test_product_far_rows(M, K, N):
    w, ws, xq, xs = operands(1, M, K, N, gen(M))
    ldx = 1 << (22 if N < 2048 else 21)
    for dtype in (torch.bfloat16, torch.float32):
        case(f"qgemm_f8 far rows M={M} K={K} N={N} {dtype}")
        Y = qg.qgemm_f8(w, ws[0], xq, xs, M, K, dtype=dtype)[:, :M]
        for ldy in (1 << 21, 1 << 22):  # (an output tile's bytes within 32 bits, and beyond)
            out = apart(torch.zeros_like(Y), ldy)
            qg.qgemm_f8(w, ws[0], apart(xq, ldx), apart(xs, 1 << 20), M, K, Y=out, dtype=dtype)
            assert torch.equal(bits(out), bits(Y)), ldy
            del out


@pytest.mark.parametrize("M,K,each", [(260, 300, 1), (260, 300, 20), (516, 700, 170), (516, 300, 170), (516, 700, 600)])
def test_grouped_far_rows(M, K, each):
    E = 3
    N = E * each
    g = gen(M + each)
    w, ws, xq, xs = operands(E, M, K, max(N, 2000), g)
    offsets = torch.tensor([0, each - each // 3, each - each // 3 + 2 * each // 3, N], dtype=torch.int32, device=DEV)
    row = torch.randint(0, xq.shape[0], (N,), generator=g, device=DEV, dtype=torch.int32)
    row[0], row[N - 1] = xq.shape[0] - 1, xq.shape[0] - 1
    far = apart(xq, 1 << 21)       # 2000 rows: just below 2^32 bytes, the most that `row` may reach into
    far_s = apart(xs, 1 << 19)
    for dtype in (torch.bfloat16, torch.float32):
        case(f"qgemm_f8_grouped far rows M={M} K={K} each={each} {dtype}")
        for r in (row, None):
            x, s = (xq, xs) if r is not None else (xq[:N], xs[:N])
            fx, fs = (far, far_s) if r is not None else (far[:N], far_s[:N])
            Y = qg.qgemm_f8_grouped(w, ws, x, s, M, K, offsets, row=r, dtype=dtype)[:, :M]
            out = apart(torch.zeros_like(Y), 1 << 22)
            qg.qgemm_f8_grouped(w, ws, fx, fs, M, K, offsets, row=r, Y=out, dtype=dtype)
            assert torch.equal(bits(out), bits(Y)), (dtype, r is None)
            del out


@pytest.mark.parametrize("N", [40, 100])
def test_select_and_combine_far_rows(N):
    case(f"logits_expert_select, expert_combine far rows N={N}")
    g = gen(N)
    z = torch.randn(N, 70, generator=g, device=DEV).half()
    a, b = qg.logits_expert_select(z, 4), qg.logits_expert_select(apart(z, 1 << 26), 4)
    for name in ("expert", "weight", "position", "row", "offsets"):
        assert torch.equal(bits(getattr(a, name)), bits(getattr(b, name))), name
    y = torch.randn(4 * N, 203, generator=g, device=DEV).bfloat16()
    add = torch.randn(N, 203, generator=g, device=DEV).bfloat16()
    o = qg.expert_combine(y, a.position, a.weight, add=add)
    out = apart(add, 1 << 26)
    qg.expert_combine(apart(y, 1 << 24), a.position, a.weight, add=out, out=out)
    assert torch.equal(bits(out), bits(o))


def test_on_two_streams_at_once():
    """Layers of other sizes on two streams, each call with its own workspace, overlapping: every result is
    that of the calls one after the other."""
    sets = []
    for i, (E, M, K, N, k) in enumerate([(16, 512, 1024, 300, 4), (24, 384, 1536, 90, 3)]):
        g = gen(100 + i)
        w, ws, _, _ = operands(E, M, K, 1, g)
        dense, dws, _, _ = operands(1, 640, K, 1, g)
        sets.append((w, ws, dense, dws[0], torch.randn(N, K, generator=g, device=DEV).bfloat16(),
                     torch.randn(N, E, generator=g, device=DEV), M, K, k))

    def layer(w, ws, dense, dws, x, z, M, K, k):
        sel = qg.logits_expert_select(z, k, normalize=True)
        xq, xs = qg.quantize_f8_rows(x)
        y = qg.qgemm_f8_grouped(w, ws, xq, xs, M, K, sel.offsets, row=sel.row, dtype=torch.bfloat16)
        return qg.expert_combine(y, sel.position, sel.weight, M=M), qg.qgemm_f8(dense, dws, xq, xs, 640, K)

    want = [layer(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for turn in range(5):
        case(f"two streams at once, turn {turn}")
        got = []
        for _ in range(4):
            for st, s in zip(streams, sets):
                with torch.cuda.stream(st):
                    got.append(layer(*s))
        torch.cuda.synchronize()
        for i, r in enumerate(got):
            for a, b in zip(r, want[i % 2]):
                assert torch.equal(bits(a), bits(b)), (turn, i)


@pytest.mark.parametrize("experts", [1, 5])
def test_products_of_more_than_4_gib_of_weights(experts):
    """The last rows of weights beyond 2^32 bytes give what they give alone."""
    M, K, last = 1200000 // experts // 256 * 256 + 44, 4096, 300
    g = gen(experts)
    codes = torch.randint(0, 120, (experts, M, K), generator=g, device=DEV, dtype=torch.uint8)
    w = codes.view(F8)
    ws = torch.rand(experts, -(-M // 128), K // 128, generator=g, device=DEV) + 0.5
    first = (M - last) // 128 * 128  # (a scale's first row)
    tail, tail_ws = qg.pack_f8(w[-1, first:]), ws[-1, first // 128:].contiguous()
    wp = qg.pack_f8(w)
    aw = w[-1, first:].double().abs() * tail_ws.double().repeat_interleave(128, 0)[:M - first].repeat_interleave(128, 1)
    for N in (2, 40, 300):
        case(f"{experts} matrices of {M} x {K} by {N}")
        xq, xs = qg.quantize_f8_rows(torch.randn(N, K, generator=g, device=DEV))
        size = (xq.double().abs() * xs.double().repeat_interleave(128, 1)[:, :K]) @ aw.t()
        for dtype in (torch.bfloat16, torch.float32):
            if experts == 1:
                y = qg.qgemm_f8(wp, ws[0], xq, xs, M, K, dtype=dtype)
            else:
                offsets = torch.tensor([0] * experts + [N], dtype=torch.int32, device=DEV)
                y = qg.qgemm_f8_grouped(wp, ws, xq, xs, M, K, offsets, dtype=dtype)
            alone = qg.qgemm_f8(tail, tail_ws, xq, xs, M - first, K, dtype=torch.float32)[:, :M - first].double()
            # a block's 128 products in float32, 32 blocks and at most 8 partial sums, on both sides in other
            # orders; on the 8-bit matrix cores 2^-10 of the terms; one rounding
            tol = size * 2 * (128 + 32 + 8) * 2.0 ** -24
            if dtype == torch.bfloat16:
                tol = (tol + size * 2.0 ** -10) * (1 + 2.0 ** -8) + alone.abs() * 2.0 ** -8
            off = (y[:, first:M].double() - alone).abs() - tol
            assert bool((off <= 0).all()), (N, dtype, float(off.max()))
            assert not bool(torch.isnan(y[:, :M]).any())
