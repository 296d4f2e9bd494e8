"""GPU parity of the products by expert with the scaled sums in 64 bits: every
scaling, format and tile size, ragged and empty segments, rows in no segment."""
import pytest
import torch

from tests import grouped_reference as G
from tests.gpu_helpers import DEV
from tests.grouped_reference import BLOCK, E2M1, MX, SQUARE, TENSOR

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def F():
    from scaled_fp8_gemm_amd import fp8sg
    fp8sg.lib()
    return fp8sg


def unwritten(*shape, dtype=BF):
    return torch.full(shape, -777.0, dtype=dtype, device=DEV)


def segments(lengths, first=0, after=0):
    """Offsets of segments one after the other, and the rows in all."""
    off = [first]
    for n in lengths:
        off.append(off[-1] + n)
    return off, off[-1] + after


def fprop(F, x, w, offsets, experts, rows, n, k, sa, sb, fa, fb, dgrad=False):
    y = unwritten(rows, n)
    xo = F.operand(x[0].to(DEV), fa, sa, x[1].to(DEV))
    wo = F.operand(w[0].to(DEV), fb, sb, w[1].to(DEV))
    off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    if dgrad:
        F.fp8_gemm_grouped_dgrad(xo, wo, off, experts, rows, k, n, y)
    else:
        F.fp8_gemm_grouped_fprop(xo, wo, off, experts, rows, n, k, y)
    return y


def some_columns(n):
    """Columns at both ends and around a tile's edge."""
    return [c for c in sorted({*range(6), *range(124, 132), *range(252, 260), *range(n - 20, n)})
            if 0 <= c < n]


def run_rows(F, orc, lengths, n, k, sa, sb, fa, fb, first=0, after=0, dgrad=False, spoil=None):
    offsets, rows = segments(lengths, first, after)
    e = len(lengths)
    x = G.operand(1 + rows, rows, k, fa, sa)
    w = G.operand(2 + n, e * n, k, fb, sb, tensors=e)
    if spoil:
        spoil(x, w)
    y = fprop(F, x, w, offsets, e, rows, n, k, sa, sb, fa, fb, dgrad)
    a = G.values(*x, fa, sa)
    b = G.values(*w, fb, sb, n if sb == TENSOR else None)
    cols = list(range(n)) if n < 600 else some_columns(n)
    for i in range(e):
        r = slice(offsets[i], offsets[i + 1])
        G.check(orc, y[r][:, cols].contiguous(), a[r], b[[i * n + c for c in cols]], f"expert {i}")
    out = torch.cat([y[:offsets[0]], y[offsets[-1]:]])
    assert (out == -777.0).all()
    return y


# (segment lengths, columns): by the mean length, and the number of tiles, the
# tiles of 16 (4-bit weights), 32, 64 rows, 64 x 128, 128 and 256, each with a
# segment longer than its tile, shorter ones and empty ones; columns that end
# inside a tile, odd ones among them
FEW16 = ([3, 0, 20, 1, 16], 70)
FEW32 = ([40, 0, 7, 33], 33)
FEW64 = ([70, 0, 64, 130, 1], 100)
WIDE64 = ([70, 0, 64, 130, 1], 1929)
MID = ([600, 1, 0, 300, 128], 3333)
BIG = ([700, 90, 513], 5381)
ALL = [FEW16, FEW32, FEW64, WIDE64, MID, BIG]


@pytest.mark.parametrize("lengths,n", ALL)
@pytest.mark.parametrize("fa,fb", [(0, 0), (1, 0), (0, 1), (1, 1)])
def test_tensor(F, orc, lengths, n, fa, fb):
    run_rows(F, orc, lengths, n, 208 if n < 600 else 144, TENSOR, TENSOR, fa, fb, first=3, after=5)


@pytest.mark.parametrize("lengths,n", ALL)
@pytest.mark.parametrize("sb", [BLOCK, SQUARE])
@pytest.mark.parametrize("fa,fb", [(0, 0), (1, 0), (0, 1), (1, 1)])
def test_block(F, orc, lengths, n, sb, fa, fb):
    n = n if sb == BLOCK else -(-n // 128) * 128
    run_rows(F, orc, lengths, n, 384 if n < 300 else 128, BLOCK, sb, fa, fb, after=9)


@pytest.mark.parametrize("lengths,n", ALL)
@pytest.mark.parametrize("k", [256, 160])
@pytest.mark.parametrize("fa,fb", [(0, 0), (1, 0), (0, 1), (1, 1), (0, E2M1), (1, E2M1),
                                   (E2M1, E2M1)])
def test_mx(F, orc, lengths, n, k, fa, fb):
    run_rows(F, orc, lengths, n, k, MX, MX, fa, fb, first=1, after=2)


# depths that end inside a step, inside 512 K, and several rounds of a
# workgroup's waves
DEEP = [([2, 5], 40), ([150], 40), ([150], 6900), ([300], 11000), ([420], 20600)]


@pytest.mark.parametrize("k", [16, 112, 640, 1040, 5136])
@pytest.mark.parametrize("lengths,n", DEEP)
def test_depths_tensor(F, orc, lengths, n, k):
    run_rows(F, orc, lengths, n, k if n < 600 else k % 1024 + 16, TENSOR, TENSOR, 0, 0)


@pytest.mark.parametrize("k", [32, 96, 384, 544, 1056, 1152, 4640, 5120])
@pytest.mark.parametrize("lengths,n", DEEP)
@pytest.mark.parametrize("fa,fb", [(0, 0), (0, E2M1), (E2M1, E2M1)])
def test_depths_mx(F, orc, lengths, n, k, fa, fb):
    run_rows(F, orc, lengths, n, k if n < 600 else k % 1024 + 32, MX, MX, fa, fb)


@pytest.mark.parametrize("k", [128, 640, 1152, 5120])
@pytest.mark.parametrize("lengths,n", [([2, 5], 128), ([150], 128), ([150], 6912), ([300], 11008),
                                       ([420], 20608)])
@pytest.mark.parametrize("sb", [BLOCK, SQUARE])
def test_depths_block(F, orc, lengths, n, k, sb):
    run_rows(F, orc, lengths, n, k if n < 600 else k % 1024 + 128, BLOCK, sb, 0, 0)


def test_dgrad(F, orc):
    run_rows(F, orc, [9, 0, 30], 48, 160, MX, MX, 1, 0, dgrad=True)
    run_rows(F, orc, [9, 0, 30], 128, 128, BLOCK, SQUARE, 1, 0, dgrad=True)


@pytest.mark.parametrize("k", [128, 160, 384, 640])
@pytest.mark.parametrize("lengths,n", [([5, 12], 40), ([60, 5], 40), ([140], 40), ([140], 6900),
                                       ([300], 11000), ([420], 20600)])
@pytest.mark.parametrize("fa,fb", [(0, 0), (0, E2M1), (E2M1, E2M1)])
def test_nan_scales_stay_in_their_row(F, orc, lengths, n, k, fa, fb):
    """A NaN scale byte makes its own row (column) NaN, and no neighbour, at
    the ends of rows too, where a step reads past them."""
    def spoil(x, w):
        x[1][1, 0] = x[1][4, -1] = 255
        w[1][2, 0] = w[1][7, -1] = w[1][-1, -1] = 255
    run_rows(F, orc, lengths, n, k, MX, MX, fa, fb, spoil=spoil)


@pytest.mark.parametrize("experts", [1, 63, 64, 65, 200, 1024])
def test_many_experts(F, orc, experts):
    g = torch.Generator().manual_seed(experts)
    lengths = torch.randint(0, 5, (experts,), generator=g).tolist()
    lengths[-1] = 21
    run_rows(F, orc, lengths, 16, 32, MX, MX, 0, E2M1)
    lengths = [0] * experts
    lengths[experts // 2] = 150 * min(experts, 70)    # all rows to one expert
    run_rows(F, orc, lengths, 16, 32, TENSOR, TENSOR, 0, 0)


def test_segments_that_are_none(F):
    """No rows, no columns, no depth; offsets outside the rows, or falling."""
    for rows, n, k in ((0, 16, 32), (5, 0, 32)):
        fprop(F, G.operand(1, rows, k, 0, MX), G.operand(2, 2 * n, k, 0, MX), [0, 0, rows], 2,
              rows, n, k, MX, MX, 0, 0)
    for rows in (5, 300):
        y = fprop(F, G.operand(1, rows, 0, 0, MX), G.operand(2, 32, 0, 0, MX), [0, 2, rows - 1], 2,
                  rows, 16, 0, MX, MX, 0, 0)
        assert (y[:rows - 1] == 0).all() and (y[rows - 1:] == -777).all()
        x, w = G.operand(1, rows, 64, 0, MX), G.operand(2, 32, 64, 0, MX)
        good = fprop(F, x, w, [0, 2, rows], 2, rows, 16, 64, MX, MX, 0, 0)
        cut = fprop(F, x, w, [-7, 2, 1 << 30], 2, rows, 16, 64, MX, MX, 0, 0)
        assert torch.equal(good, cut)
        assert (fprop(F, x, w, [4, 2, 1], 2, rows, 16, 64, MX, MX, 0, 0) == -777).all()


# ------------------------------------------------------------ weight gradients
def run_depth(F, orc, lengths, n, k, scaling, fa, fb, out="bf16", after=0, unit=128):
    offsets, rows = segments([v * unit for v in lengths], 0, after * unit)
    e = len(lengths)
    a, b = G.operand(3 + rows, n, rows, fa, scaling), G.operand(4 + k, k, rows, fb, scaling)
    ao = F.operand(a[0].to(DEV), fa, scaling, a[1].to(DEV))
    bo = F.operand(b[0].to(DEV), fb, scaling, b[1].to(DEV))
    off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    old = torch.zeros(e, n, k)
    if out == "bf16":
        dw = unwritten(e, n, k) * float("nan")
        F.fp8_gemm_grouped_wgrad(ao, bo, off, e, rows, n, k, dw)
    else:
        dw = unwritten(e, n, k, dtype=torch.float32) * float("nan")
        if out == "add":
            old = torch.randn(e, n, k, generator=torch.Generator().manual_seed(9))
            dw.copy_(old)
        F.fp8_gemm_grouped_wgrad_f32(ao, bo, off, e, rows, n, k, dw, accumulate=out == "add")
    av, bv = G.values(*a, fa, scaling), G.values(*b, fb, scaling)
    m, c = (some_columns(n), some_columns(k)) if n * k > 1 << 20 else (range(n), range(k))
    av, bv = av[list(m)], bv[list(c)]
    got, old = dw[:, list(m)][:, :, list(c)], old[:, list(m)][:, :, list(c)]
    for i in range(e):
        r = slice(offsets[i], offsets[i + 1])
        if out == "bf16":
            G.check(orc, got[i].contiguous(), av[:, r], bv[:, r], f"expert {i}")
        else:
            G.check_f32(got[i], old[i], av[:, r], bv[:, r], f"expert {i}")
    assert not dw.isnan().any()                      # every output written
    return dw


@pytest.mark.parametrize("scaling", [TENSOR, BLOCK, MX])
@pytest.mark.parametrize("fa,fb", [(0, 0), (1, 0), (0, 1), (1, 1)])
@pytest.mark.parametrize("out", ["bf16", "f32", "add"])
def test_wgrad(F, orc, scaling, fa, fb, out):
    run_depth(F, orc, [2, 0, 1, 5], 130, 71, scaling, fa, fb, out, after=1)


@pytest.mark.parametrize("n,k", [(1, 1), (16, 264), (257, 8), (300, 72)])
def test_wgrad_sizes(F, orc, n, k):
    run_depth(F, orc, [1, 0, 3], n, k, MX, 0, 0)
    run_depth(F, orc, [3, 1, 0, 9], n, k, TENSOR, 1, 0, unit=16, after=3)


# whole float4s of an FP32 result in tiles of 64; tiles of 256, with rows of any
# length too; results that are written past the caches
@pytest.mark.parametrize("lengths,n,k", [([2, 0, 1, 5], 130, 72), ([2, 0, 1, 3, 1, 0, 1, 1], 1300, 1616),
                                         ([2, 0, 1, 1, 1, 0, 1, 1], 1300, 1615),
                                         ([0, 1, 1, 0, 1, 0, 2, 1], 2900, 2904)])
@pytest.mark.parametrize("scaling,fa,fb", [(TENSOR, 1, 0), (TENSOR, 0, 0), (BLOCK, 0, 1), (MX, 0, 0),
                                           (MX, 1, 1)])
@pytest.mark.parametrize("out", ["bf16", "f32", "add"])
def test_wgrad_tiles(F, orc, lengths, n, k, scaling, fa, fb, out):
    run_depth(F, orc, lengths, n, k, scaling, fa, fb, out, after=1)


@pytest.mark.parametrize("sa,fb", [(TENSOR, 0), (BLOCK, 0), (MX, E2M1)])
def test_rows_written_past_the_caches(F, orc, sa, fb):
    run_rows(F, orc, [700, 90, 513], 52104, 128, sa, sa, 0, fb, after=5)


def test_wgrad_without_rows(F):
    dw = run_depth(F, None, [0, 0], 0, 0, MX, 0, 0)
    assert dw.numel() == 0
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    e = torch.empty(0, dtype=torch.uint8, device=DEV)
    dw = unwritten(2, 40, 24)
    op = F.operand(e, 0, MX, torch.empty(4, dtype=torch.uint8, device=DEV))
    F.fp8_gemm_grouped_wgrad(op, op, off, 2, 0, 40, 24, dw)
    assert (dw == 0).all()
    acc = unwritten(2, 40, 24, dtype=torch.float32)
    F.fp8_gemm_grouped_wgrad_f32(op, op, off, 2, 0, 40, 24, acc, accumulate=True)
    assert (acc == -777).all()


def test_nan_scales_of_other_segments(F, orc):
    """A NaN scale of one expert's rows is none of another's."""
    a, b = G.operand(1, 20, 512, 0, MX), G.operand(2, 24, 512, 0, MX)
    a[1][3, 4], b[1][5, 11] = 255, 255               # rows 128 .. 383: expert 1
    off = torch.tensor([0, 128, 384, 512], dtype=torch.int32, device=DEV)
    dw = unwritten(3, 20, 24)
    F.fp8_gemm_grouped_wgrad(F.operand(a[0].to(DEV), 0, MX, a[1].to(DEV)),
                             F.operand(b[0].to(DEV), 0, MX, b[1].to(DEV)), off, 3, 512, 20, 24, dw)
    bad = torch.isnan(dw.cpu())
    assert not bad[0].any() and not bad[2].any()
    assert bad[1, 3].all() and bad[1, :, 5].all() and int(bad[1].sum()) == 24 + 20 - 1


# ------------------------------------------------------------ as it is used
@pytest.mark.parametrize("lengths", [[3, 0, 20, 9], [300, 129, 0, 200]])
def test_captured_with_offsets_of_each_replay(F, orc, lengths):
    """The segments are read at replay: other offsets, other results, equal to
    the eager calls', with eager work between the replays."""
    e, n, k = 4, 72, 160
    offsets, rows = segments(lengths)
    rows = -(-rows // 128) * 128
    x, w = G.operand(5, rows, k, 0, MX), G.operand(6, e * n, k, 0, MX)
    xt, yt = G.operand(7, n, rows, 0, MX), G.operand(8, k, rows, 0, MX)
    ops = [F.operand(q.to(DEV), 0, MX, s.to(DEV)) for q, s in (x, w, xt, yt)]
    off = torch.zeros(e + 1, dtype=torch.int32, device=DEV)

    def both(y, dw, stream=None):
        F.fp8_gemm_grouped_fprop(ops[0], ops[1], off, e, rows, n, k, y, stream=stream)
        F.fp8_gemm_grouped_wgrad(ops[2], ops[3], off, e, rows, n, k, dw, stream=stream)
    y, dw, graph = unwritten(rows, n), unwritten(e, n, k), torch.cuda.CUDAGraph()
    both(y, dw)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        both(y, dw)
    side = torch.cuda.Stream()
    for i in range(4):
        new = [v // 128 * 128 for v in offsets] if i % 2 else [0, 0, 128 * (i // 2), 128, rows]
        off.copy_(torch.tensor(new, dtype=torch.int32))
        y.fill_(-777)
        graph.replay()
        y2, dw2 = unwritten(rows, n), unwritten(e, n, k)
        torch.cuda.synchronize()
        both(y2, dw2, side)
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(dw, dw2), i


def test_offsets_from_the_sort(F, orc):
    """fp8_moe_sort's offsets and fp8_moe_dispatch's operand, as they come."""
    tokens, k, e, c, n = 37, 2, 5, 96, 40
    g = torch.Generator().manual_seed(1)
    x = torch.randn(tokens, c, generator=g).bfloat16().to(DEV)
    expert = torch.randint(-1, e, (tokens, k), generator=g).int().to(DEV)
    rows = F.moe_rows(tokens * k, e, 16)
    i32 = lambda *s: torch.empty(s, dtype=torch.int32, device=DEV)  # noqa: E731
    off, cnt, pos, src = i32(e + 1), i32(e), i32(tokens, k), i32(rows)
    F.fp8_moe_sort(expert, e, 16, off, cnt, pos, src)
    q = torch.empty(rows, c, dtype=torch.uint8, device=DEV)
    s = torch.empty(rows, c // 32, dtype=torch.uint8, device=DEV)
    F.fp8_moe_dispatch(x, pos, src, off, None, xq=F.cast_out(q, 0, MX, s))
    w = G.operand(2, e * n, c, E2M1, MX)
    y = unwritten(rows, n)
    F.fp8_gemm_grouped_fprop(F.operand(q, 0, MX, s),
                             F.operand(w[0].to(DEV), E2M1, MX, w[1].to(DEV)), off, e, rows, n, c, y)
    at = off.tolist()
    a, b = G.values(q, s, 0, MX), G.values(*w, E2M1, MX)
    for i in range(e):
        r = slice(at[i], at[i + 1])
        G.check(orc, y[r], a[r], b[i * n:(i + 1) * n], f"expert {i}")
        assert (y[at[i] + int(cnt[i]):at[i + 1]] == 0).all()        # padding
    assert (y[at[-1]:] == -777).all()


@pytest.mark.parametrize("lengths", [[3, 6], [300, 500]])
def test_more_than_2_31_elements(F, orc, lengths):
    """Weights and outputs past 2^31 elements, by their last rows and columns."""
    if lengths[0] < 10:
        n, k = 40000, 32768                        # 2.6 10^9 weights
    else:
        lengths, n, k = [66000, 300], 33000, 32    # 2.2 10^9 outputs
    offsets, rows = segments(lengths)
    g = torch.Generator(device=DEV).manual_seed(3)
    byte = lambda hi, *s: torch.randint(0, hi, s, generator=g, device=DEV, dtype=torch.uint8)  # noqa: E731
    x, xs = byte(0x7f, rows, k), torch.full((rows, k // 32), 120, dtype=torch.uint8, device=DEV)
    w, ws = byte(256, 2 * n, k // 2), 120 + byte(8, 2 * n, k // 32)
    y = torch.empty(rows, n, dtype=BF, device=DEV)
    F.fp8_gemm_grouped_fprop(F.operand(x, 0, MX, xs), F.operand(w, E2M1, MX, ws),
                             torch.tensor(offsets, dtype=torch.int32, device=DEV), 2, rows, n, k, y)
    a, b = G.values(x[-3:], xs[-3:], 0, MX), G.values(w[-5:], ws[-5:], E2M1, MX)
    G.check(orc, y[-3:, -5:].contiguous(), a, b, "last")


def test_more_tiles_than_a_grid(F, orc):
    """1024 experts of one row and so many columns that the small tiles which
    one row would have are more than a grid: every expert's row, at both ends
    of the columns and at tiles' edges."""
    experts, n, k = 1024, 262400, 16
    g = torch.Generator(device=DEV).manual_seed(4)
    w = torch.randint(0, 64, (experts, n, k), generator=g, device=DEV, dtype=torch.uint8)
    x = torch.randint(0, 64, (experts, k), generator=g, device=DEV, dtype=torch.uint8)
    sx, sw = torch.ones(1, device=DEV), torch.full((experts,), 0.5, device=DEV)
    off = torch.arange(experts + 1, dtype=torch.int32, device=DEV)
    y = unwritten(experts, n) * float("nan")
    F.fp8_gemm_grouped_fprop(F.operand(x, 0, TENSOR, sx), F.operand(w, 0, TENSOR, sw), off,
                             experts, experts, n, k, y)
    cols = some_columns(n)
    some, a = w[:, cols].cpu(), G.values(x, sx, 0, TENSOR)
    got = y[:, cols].cpu()
    for e in (0, 1, 500, 1022, 1023):
        b = G.values(some[e], sw[:1].cpu(), 0, TENSOR)
        G.check(orc, got[e:e + 1].to(DEV), a[e:e + 1], b, f"expert {e}")
    assert not y.isnan().any()                       # every output written
