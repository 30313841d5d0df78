"""The product in 8-bit integers vs its definition.

Tolerances, from the arithmetic: quantisation is IEEE float32 (an absolute
maximum, a quotient by 127, quotients rounded to nearest even), which numpy's
float32 operations are too: bit for bit.  The product's sum is an exact integer;
it is converted to fp32 (2^-24), multiplied by two scales (2^-24 each) and
rounded to the output type (half a step).  A log-sum-exp moves by at most the
largest error of its logits, plus the fp32 sum: at most 256 sequential terms
per tile and one per 32 tiles (2^-24 each), exponentials of 2^-22, and the
rounding of the arguments and the result (2^-23 of their size)."""
import numpy as np
import pytest
import torch

from trie_constrained_beam_fr_b200 import fr

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def _padded(rows, cols, dtype, quantum, extra=0):
    t = torch.empty(rows, -(-cols // quantum) * quantum + extra, dtype=dtype, device="cuda")
    if dtype == torch.int8:
        t.fill_(77)  # what lies between the rows must not matter
    return t[:, :cols]


def _ints(g, rows, d, extra=0):
    q = _padded(rows, d, torch.int8, 16, extra)
    q.copy_(torch.randint(-127, 128, (rows, d), generator=g, dtype=torch.int32).to(torch.int8))
    return q


def _product(xq, xs, wq, ws):
    acc = xq.double().cpu() @ wq.double().cpu().T  # exact
    return acc * xs.double().cpu()[:, None] * ws.double().cpu()


@pytest.fixture
def handle():
    made = []

    def make(*a, **k):
        made.append(fr.fr_i8_init(*a, **k))
        return made[-1]

    yield make
    for h in made:
        fr.fr_i8_destroy(h)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,d,pad", [(1, 1, 0), (3, 15, 0), (9, 64, 0), (33, 257, 0), (100, 2048, 0), (5, 9001, 0), (17, 40, 3)])
def test_quantize(dtype, rows, d, pad):
    g = torch.Generator().manual_seed(rows * 31 + d)
    x = _padded(rows, d + pad, dtype, 1)[:, :d]
    x.copy_(torch.randn(rows, d, generator=g) * torch.exp(torch.randn(rows, 1, generator=g) * 3))
    if rows > 2:
        x[1] = 0.0
        x[2, 0] = 0.0
    if d > 8:  # values that fall between two steps, exactly
        x[0] = 0.5
        x[0, 0] = 127.0
        x[0, 1], x[0, 2], x[0, 3] = 1.5, -2.5, -126.5
    q, s = torch.full((rows, d + 5), 99, dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    fr.fr_i8_quantize(x, q[:, :d], s)
    # numpy's float32 quotients are IEEE (torch divides by a number through its reciprocal)
    xf = x.float().cpu().numpy()
    want_s = np.abs(xf).max(1) / np.float32(127)
    want = np.rint(xf / np.where(want_s > 0, want_s, np.float32(1))[:, None])
    assert np.array_equal(s.cpu().numpy(), want_s)
    assert np.array_equal(q[:, :d].cpu().numpy(), want.astype(np.int8))
    assert torch.all(q[:, d:] == 99)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_quantize_near_halves(dtype):
    """Values on and next to the borders between two steps, at scales from
    subnormal to large: the rounded IEEE quotients, bit for bit."""
    g = torch.Generator().manual_seed(2)
    rows, d = 400, 1024
    x = torch.empty(rows, d)
    top = torch.exp2(torch.linspace(-146, 127, rows))[:, None] * (1 + torch.rand(rows, 1, generator=g))
    top = torch.where(torch.isfinite(top), top, torch.full_like(top, 3e38))
    half = (torch.randint(-127, 127, (rows, d), generator=g) + 0.5) / 127
    x = half.double() * top.double() * (1 + torch.randint(-3, 4, (rows, d), generator=g).double() * 2.0 ** -24)
    x[:, 0] = top[:, 0].double()
    x = x.float().to(dtype).cuda()
    q, s = torch.empty(rows, d, dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    fr.fr_i8_quantize(x, q, s)
    xf = x.float().cpu().numpy()
    want_s = np.abs(xf).max(1) / np.float32(127)
    live = want_s > 0  # below 127 subnormal steps the scale itself may round to zero
    want = np.clip(np.rint(xf / np.where(live, want_s, np.float32(1))[:, None]), -127, 127) * live[:, None]
    assert np.array_equal(s.cpu().numpy(), want_s)
    assert np.array_equal(q.cpu().numpy(), want.astype(np.int8))


def test_quantize_rows_that_are_not_finite():
    x = torch.ones(3, 40, device="cuda")
    x[0, 7], x[1, 39] = float("nan"), float("-inf")
    q, s = torch.empty(3, 40, dtype=torch.int8, device="cuda"), torch.empty(3, device="cuda")
    fr.fr_i8_quantize(x, q, s)
    assert torch.isnan(s[0]) and torch.isinf(s[1]) and s[2] == np.float32(1) / np.float32(127)
    assert torch.all(q[:2] == 0) and torch.all(q[2] == 127)


# one or two long rows stream the weight; the others run on tiles of 64 to 256 columns
SHAPES = [(1, 1, 1), (1, 300, 9000), (2, 77, 1537), (1, 2001, 1600), (2, 130, 30000), (2, 130, 40000), (1, 300, 64), (2, 77, 130), (3, 2001, 1000), (4, 41, 7), (4, 300, 9000), (4, 130, 20000), (5, 1000, 2048), (9, 130, 50),
          (16, 513, 96), (20, 15001, 40), (33, 64, 16), (100, 1003, 521), (128, 256, 128),
          (129, 2500, 333), (300, 700, 4096)]


@pytest.mark.parametrize("tout", [F32, BF16])
@pytest.mark.parametrize("rows,N,d", SHAPES)
def test_matmul(handle, tout, rows, N, d):
    g = torch.Generator().manual_seed(rows + N + d)
    xq, wq = _ints(g, rows, d), _ints(g, N, d, extra=16)
    xs, ws = torch.rand(rows, generator=g).cuda(), torch.rand(N, generator=g).cuda()
    h = handle(wq, ws, rows)
    for pad in (0, 3):  # rows that start on 16 bytes or not
        out = torch.full((rows, N + pad), 5.0, dtype=tout, device="cuda")
        fr.fr_i8_matmul(h, xq, xs, out[:, :N])
        assert fr.fr_i8_status(h) == fr.FR_OK
        want = _product(xq, xs, wq, ws)
        err = (out[:, :N].double().cpu() - want).abs()
        assert torch.all(err <= (3.1 * 2.0 ** -24 + torch.finfo(tout).eps / 2) * want.abs())
        assert torch.all(out[:, N:] == 5.0)


@pytest.mark.parametrize("value", [-128, 127])
def test_the_largest_sums(handle, value):
    """All values at the end of the range, at the largest d a few rows allow."""
    d = 131056
    xq, wq = _padded(2, d, torch.int8, 16), _padded(20, d, torch.int8, 16)
    xq.fill_(value), wq.fill_(-128)
    h = handle(wq, torch.ones(20, device="cuda"), 2)
    out = torch.empty(2, 20, device="cuda")
    fr.fr_i8_matmul(h, xq, torch.ones(2, device="cuda"), out)
    want = float(value * -128 * d)
    assert torch.all((out.double() - want).abs() <= 2.0 ** -24 * abs(want))


@pytest.mark.parametrize("rows,N,d,base,span", [(1, 64, 32, 0, 64), (3, 300, 64, 100, 37), (40, 1000, 520, 990, 10), (130, 700, 256, 200, 0),
                                                (300, 5000, 96, 0, 768), (300, 1500, 200, 77, 1301), (33, 2000, 257, 129, 640),
                                                (20, 40000, 64, 39000, 1000), (300, 16500, 40, 1, 90)])
def test_lse(handle, rows, N, d, base, span):
    g = torch.Generator().manual_seed(rows + N)
    xq, wq = _ints(g, rows, d), _ints(g, N, d)
    xs = (torch.rand(rows, generator=g) / 73 + 1e-4).cuda()
    ws = (torch.rand(N, generator=g) / 73 * 3 / d ** 0.5).cuda()
    h = handle(wq, ws, rows, base, span)
    lse, sl = torch.empty(rows, device="cuda"), torch.empty(rows, span, device="cuda")
    fr.fr_i8_lse(h, xq, xs, lse, sl if span else None)
    assert fr.fr_i8_status(h) == fr.FR_OK
    y = _product(xq, xs, wq, ws)
    want = torch.logsumexp(y, 1)
    big = y.abs().amax(1)
    bound = 3.1 * 2.0 ** -24 * big + (256 + N / 8192 + 8) * 2.0 ** -24 + 2.0 ** -22 + 2.0 ** -23 * (want.abs() + 3 * big)
    assert torch.all((lse.double().cpu() - want).abs() <= bound)
    assert torch.all((sl.double().cpu() - y[:, base:base + span]).abs() <= 3.1 * 2.0 ** -24 * y[:, base:base + span].abs())


@pytest.mark.parametrize("rows", [3, 40, 140])
@pytest.mark.parametrize("d", [255, 256, 257])
def test_sums_at_the_end_of_the_short_rows(handle, rows, d):
    """Sums of short rows (up to 2^22) and of longer ones are converted in two
    ways: exact at the border, with values at both ends of the range."""
    xq, wq = _padded(rows, d, torch.int8, 16), _padded(70, d, torch.int8, 16)
    xq.fill_(-128), wq.fill_(-128)
    xq[1], wq[1::2] = 127, 127
    xq[2, ::2] = 0
    h = handle(wq, torch.ones(70, device="cuda"), rows, 3, 64)
    xs, out = torch.ones(rows, device="cuda"), torch.empty(rows, 70, device="cuda")
    fr.fr_i8_matmul(h, xq, xs, out)
    want = _product(xq, xs, wq, torch.ones(70))
    assert torch.equal(out.double().cpu(), want)
    lse, sl = torch.empty(rows, device="cuda"), torch.empty(rows, 64, device="cuda")
    fr.fr_i8_lse(h, xq, xs, lse, sl)
    assert torch.equal(sl.double().cpu(), want[:, 3:67])


@pytest.mark.parametrize("rows", [1, 2, 3])
@pytest.mark.parametrize("N,d", [(5, 16), (5, 17), (8, 527), (9, 2048), (9, 2049), (10, 2063), (31, 2064), (6, 5000), (6, 6143)])
def test_the_few_rows_last_pieces(handle, rows, N, d):
    """Rows that end anywhere in the pieces, and a weight that ends with its last row."""
    g = torch.Generator().manual_seed(N * d)
    xq, pitch = _ints(g, rows, d), -(-d // 16) * 16
    flat = torch.randint(-127, 128, ((N - 1) * pitch + d,), generator=g, dtype=torch.int32).to(torch.int8).cuda()
    wq = flat.as_strided((N, d), (pitch, 1))
    h = handle(wq, torch.ones(N, device="cuda"), rows)
    xs, out = torch.ones(rows, device="cuda"), torch.empty(rows, N, device="cuda")
    fr.fr_i8_matmul(h, xq, xs, out)
    want = _product(xq, xs, wq, torch.ones(N))
    assert torch.all((out.double().cpu() - want).abs() <= 2.0 ** -24 * want.abs())


def test_a_row_that_is_not_finite_is_recorded(handle):
    g = torch.Generator().manual_seed(1)
    wq = _ints(g, 50, 32)
    h = handle(wq, torch.ones(50, device="cuda"), 4, 0, 8)
    xq, xs = _ints(g, 4, 32), torch.tensor([1e-3, float("nan"), 1e-3, 1e-3], device="cuda")
    lse, sl = torch.empty(4, device="cuda"), torch.empty(4, 8, device="cuda")
    fr.fr_i8_lse(h, xq, xs, lse, sl)
    assert fr.fr_i8_status(h) == fr.FR_ERR_NAN_LOGIT
    assert torch.isnan(lse[1]) and torch.all(torch.isfinite(lse[[0, 2, 3]]))
    fr.fr_i8_clear_status(h)
    assert fr.fr_i8_status(h) == fr.FR_OK


def test_fewer_rows_and_none(handle):
    g = torch.Generator().manual_seed(4)
    wq = _ints(g, 70, 48)
    h = handle(wq, torch.ones(70, device="cuda"), 200)
    xq, xs = _ints(g, 200, 48), torch.rand(200, generator=g).cuda()
    whole = torch.empty(200, 70, device="cuda")
    fr.fr_i8_matmul(h, xq, xs, whole)
    for n in (0, 1, 37, 128):
        out = torch.full((200, 70), 3.0, device="cuda")
        fr.fr_i8_matmul(h, xq[:n], xs[:n], out[:n])
        assert torch.equal(out[:n], whole[:n]) and torch.all(out[n:] == 3.0)


def test_graph_and_another_stream(handle):
    g = torch.Generator().manual_seed(8)
    N, d, rows = 900, 200, 150
    wq = _ints(g, N, d)
    h = handle(wq, torch.rand(N, generator=g).cuda() / 100, rows, 17, 100)
    x = torch.randn(rows, d, generator=g).to(BF16).cuda()
    xq, xs = _padded(rows, d, torch.int8, 16), torch.empty(rows, device="cuda")
    lse, sl, out = torch.empty(rows, device="cuda"), torch.empty(rows, 100, device="cuda"), torch.empty(rows, N, device="cuda")

    def run():
        fr.fr_i8_quantize(x, xq, xs)
        fr.fr_i8_lse(h, xq, xs, lse, sl)
        fr.fr_i8_matmul(h, xq, xs, out)

    run()
    want = [t.clone() for t in (lse, sl, out)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        run()
    for _ in range(2):
        for t in (lse, sl, out):
            t.fill_(9.0)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip((lse, sl, out), want))
    with torch.cuda.stream(s):
        s.wait_stream(torch.cuda.default_stream())
        out.fill_(9.0)
        run()
    s.synchronize()
    assert torch.equal(out, want[2])


def test_a_wait_that_expires(handle):
    """The producer issues no copies: the product gives up after 1 ms, records
    it, and the handle works again afterwards."""
    g = torch.Generator().manual_seed(6)
    wq = _ints(g, 600, 256)
    h = handle(wq, torch.ones(600, device="cuda"), 200)
    xq, xs, out = _ints(g, 200, 256), torch.ones(200, device="cuda"), torch.empty(200, 600, device="cuda")
    fr.fr_i8_set_wait_test(h, 1_000_000, True)
    fr.fr_i8_matmul(h, xq, xs, out)
    assert fr.fr_i8_status(h) == fr.FR_ERR_DEVICE
    fr.fr_i8_set_wait_test(h, 0, False)
    fr.fr_i8_clear_status(h)
    fr.fr_i8_matmul(h, xq, xs, out)
    assert fr.fr_i8_status(h) == fr.FR_OK
    assert torch.equal(out.double().cpu(), _product(xq, xs, wq, torch.ones(600)))


def test_refusals(handle):
    g = torch.Generator().manual_seed(3)
    wq, ws = _ints(g, 40, 32), torch.ones(40, device="cuda")
    with pytest.raises(fr.FrError):
        fr.fr_i8_init(wq, ws, 4, 30, 20)  # SID range past N
    with pytest.raises(fr.FrError):
        fr.fr_i8_init(torch.zeros(40, 40, dtype=torch.int8, device="cuda"), ws, 4)  # pitch not a multiple of 16
    with pytest.raises(ValueError):
        fr.fr_i8_init(wq, ws[:39], 4)
    h = handle(wq, ws, 4, 0, 8)
    xq, xs, out = _ints(g, 4, 32), torch.ones(4, device="cuda"), torch.ones(4, 40, device="cuda")
    for bad in (lambda: fr.fr_i8_matmul(h, xq[:, :31], xs, out), lambda: fr.fr_i8_matmul(h, xq, xs[:3], out),
                lambda: fr.fr_i8_matmul(h, xq, xs, out[:, :39]), lambda: fr.fr_i8_matmul(h, xq.float(), xs, out),
                lambda: fr.fr_i8_matmul(h, xq, xs, out.half()), lambda: fr.fr_i8_lse(h, xq, xs, xs, None),
                lambda: fr.fr_i8_lse(h, xq, xs, xs, out[:, :8]), lambda: fr.fr_i8_quantize(xq, xq, xs)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(fr.FrError):
        fr.fr_i8_matmul(h, _ints(g, 5, 32), torch.ones(5, device="cuda"), torch.ones(5, 40, device="cuda"))  # > max_rows
    with pytest.raises(fr.FrError):  # base not on 16 bytes
        fr.fr_i8_matmul(h, torch.zeros(4 * 32 + 1, dtype=torch.int8, device="cuda")[1:].view(4, 32), xs, out)


# A tile of 256 columns is taken where that fills the pairs' rounds (74 pairs on 148
# SMs), and more than 8,192 rows are walked in groups of 32 tile rows.
WIDE = [(300, 9472, 64), (257, 9410, 300), (512, 9345, 128), (9000, 1000, 48), (8500, 2050, 272)]


@pytest.mark.parametrize("tout", [F32, BF16])
@pytest.mark.parametrize("rows,N,d", WIDE)
def test_matmul_of_whole_tiles_and_groups(handle, tout, rows, N, d):
    g = torch.Generator().manual_seed(rows + N + d)
    xq, wq = _ints(g, rows, d), _ints(g, N, d, extra=16)
    xs, ws = torch.rand(rows, generator=g).cuda(), torch.rand(N, generator=g).cuda()
    h = handle(wq, ws, rows)
    want = _product(xq, xs, wq, ws)
    for pad in (0, 3, 8):  # rows that start on 16 bytes or not
        out = torch.full((rows, N + pad), 5.0, dtype=tout, device="cuda")
        fr.fr_i8_matmul(h, xq, xs, out[:, :N])
        assert fr.fr_i8_status(h) == fr.FR_OK
        err = (out[:, :N].double().cpu() - want).abs()
        assert torch.all(err <= (3.1 * 2.0 ** -24 + torch.finfo(tout).eps / 2) * want.abs())
        assert torch.all(out[:, N:] == 5.0)


@pytest.mark.parametrize("rows,N,d,base,span", [(300, 9472, 64, 200, 700), (257, 9410, 300, 9310, 100), (512, 9345, 128, 0, 0),
                                                (9000, 1000, 48, 250, 300), (8500, 2050, 272, 2049, 1)])
def test_lse_of_whole_tiles_and_groups(handle, rows, N, d, base, span):
    g = torch.Generator().manual_seed(rows + N)
    xq, wq = _ints(g, rows, d), _ints(g, N, d)
    xs = (torch.rand(rows, generator=g) / 73 + 1e-4).cuda()
    ws = (torch.rand(N, generator=g) / 73 * 3 / d ** 0.5).cuda()
    h = handle(wq, ws, rows, base, span)
    lse, sl = torch.empty(rows, device="cuda"), torch.empty(rows, span, device="cuda")
    fr.fr_i8_lse(h, xq, xs, lse, sl if span else None)
    assert fr.fr_i8_status(h) == fr.FR_OK
    y = _product(xq, xs, wq, ws)
    want = torch.logsumexp(y, 1)
    big = y.abs().amax(1)
    bound = 3.1 * 2.0 ** -24 * big + (256 + N / 8192 + 8) * 2.0 ** -24 + 2.0 ** -22 + 2.0 ** -23 * (want.abs() + 3 * big)
    assert torch.all((lse.double().cpu() - want).abs() <= bound)
    assert torch.all((sl.double().cpu() - y[:, base:base + span]).abs() <= 3.1 * 2.0 ** -24 * y[:, base:base + span].abs())
