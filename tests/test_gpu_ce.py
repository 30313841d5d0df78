"""Cross entropy of the lm_head projection and its gradients vs the formulas
in double.

Tolerances, from the arithmetic.  A logit is a d-term dot product of bf16
values (exact products) accumulated in fp32: its error is at most
D = d * 2^-23 * sum |h w|.  The log-sum-exp moves by at most the largest D of
its row, plus the fp32 sum of exponentials: at most 256 sequential terms per
tile and one per 32 tiles (2^-24 each), exponentials of 2^-22, and the
rounding of their arguments and of the result (2^-23 of the values' size).
The gradient's G = g (p - [v = t]) has the error of x and lse in p (relative),
and is rounded to bf16 (half a step, 2^-8); the sums over V or over the rows
add (terms) * 2^-23 of the sum of magnitudes, and the output is rounded to
bf16 once more."""
import pytest
import torch

from trie_constrained_beam_fr_b200 import fr

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _padded(rows, cols, extra=0):
    """bf16 [rows, cols] whose pitch is a multiple of 8 elements; NaN between the rows."""
    t = torch.full((rows, -(-cols // 8) * 8 + extra), float("nan"), dtype=BF16, device="cuda")
    return t[:, :cols]


def _inputs(rows, V, d, seed, gain=2.0, ignored=0.2, extra=0):
    g = torch.Generator().manual_seed(seed)
    h, w = _padded(rows, d, extra), _padded(V, d, extra)
    h.copy_(torch.randn(rows, d, generator=g))
    w.copy_(torch.randn(V, d, generator=g) * gain / d ** 0.5)
    t = torch.randint(0, V, (rows,), generator=g, dtype=torch.int32)
    t[torch.rand(rows, generator=g) < ignored] = -1
    gl = torch.rand(rows, generator=g) * 2 - 0.5
    return h, w, t.cuda(), gl.cuda()


def _reference(h, w, t, gl):
    h, w, t, gl = h.double().cpu(), w.double().cpu(), t.long().cpu(), gl.double().cpu()
    live = t >= 0
    h = torch.where(live[:, None], h, 0.0)
    d, V, n = h.shape[1], w.shape[0], max(1, int(live.sum()))
    x = h @ w.T
    D = d * 2.0 ** -23 * (h.abs() @ w.abs().T)
    big = x.abs().amax(1)
    lse = torch.logsumexp(x, 1)
    b_lse = D.amax(1) + (256 + V / 8192 + 8) * 2.0 ** -24 + 2.0 ** -22 + 2.0 ** -23 * (lse.abs() + 3 * big)
    at = t.clamp(min=0)[:, None]
    loss = lse - x.gather(1, at)[:, 0]
    b_loss = b_lse + D.gather(1, at)[:, 0] + 2.0 ** -24 * loss.abs()
    p = torch.exp(x - lse[:, None])
    hot = torch.zeros_like(p).scatter_(1, at, 1.0)
    gl = torch.where(live, gl, 0.0)
    G = (p - hot) * gl[:, None]
    b_p = p * torch.expm1(D + (b_lse + 2.0 ** -22 + 2.0 ** -23 * (lse.abs() + big))[:, None])
    b_G = (b_p + 2.0 ** -23 * (p + hot)) * gl.abs()[:, None]
    b_G = b_G + 2.0 ** -8 * (G.abs() + b_G)
    m = G.abs() + b_G
    dh, dw = G @ w, G.T @ h
    b_dh = b_G @ w.abs() + V * 2.0 ** -23 * (m @ w.abs())
    b_dw = b_G.T @ h.abs() + n * 2.0 ** -23 * (m.T @ h.abs())
    zero = torch.zeros_like(lse)
    return dict(lse=(torch.where(live, lse, zero), b_lse), loss=(torch.where(live, loss, zero), b_loss),
                dh=(dh, b_dh + 2.0 ** -8 * (dh.abs() + b_dh)), dw=(dw, b_dw + 2.0 ** -8 * (dw.abs() + b_dw)))


def _close(got, ref):
    want, bound = ref
    err = (got.double().cpu() - want).abs()
    assert torch.all(err <= bound), "largest error over its bound: %.3g" % float((err / bound.clamp(min=1e-300)).max())


@pytest.fixture
def handle():
    made = []

    def make(*a):
        made.append(fr.fr_ce_init(*a))
        return made[-1]

    yield make
    for h in made:
        fr.fr_ce_destroy(h)


def _loss(ce, h, w, t):
    loss, lse = torch.full((len(t),), 7.0, device="cuda"), torch.full((len(t),), 7.0, device="cuda")
    fr.fr_ce_loss(ce, h, w, t, loss, lse)
    return loss, lse


def _grad(ce, h, w, t, lse, gl, pad=0, offset=0):
    """Gradients into tensors whose rows start `offset` elements into their
    storage, `pad` elements apart; checks that nothing else was written."""
    outs = []
    for rows in (h.shape[0], w.shape[0]):
        d = h.shape[1]
        flat = torch.full((rows * (d + pad) + offset + 8,), 5.0, dtype=BF16, device="cuda")
        outs.append(flat[offset:offset + rows * (d + pad)].view(rows, d + pad)[:, :d])
    fr.fr_ce_grad(ce, h, w, t, lse, gl, *outs)
    for o in outs:
        mask = torch.ones_like(o._base, dtype=torch.bool)
        mask[offset:offset + o.shape[0] * (o.shape[1] + pad)].view(o.shape[0], o.shape[1] + pad)[:, :o.shape[1]] = False
        assert torch.all(o._base[mask] == 5.0)
    return outs


@pytest.mark.parametrize("rows,V,d,ignored,gain,pad,offset", [
    (1, 1, 1, 0.0, 1.0, 0, 0),
    (1, 300, 64, 0.0, 2.0, 0, 0),
    (5, 64, 8, 0.2, 2.0, 0, 0),
    (130, 257, 72, 0.3, 2.0, 3, 1),
    (300, 1000, 200, 0.5, 2.0, 8, 8),
    (128, 256, 256, 0.0, 2.0, 0, 0),
    (129, 8500, 64, 0.0, 2.0, 0, 0),     # two pieces of the vocabulary
    (64, 20000, 137, 0.1, 2.0, 0, 0),    # three pieces, an odd hidden size, few rows
    (700, 3000, 520, 0.1, 30.0, 0, 0),   # peaked rows: probabilities near 0 and 1
    (260, 16400, 264, 0.9, 2.0, 5, 0),   # most rows do not count; last piece of 16 tokens
    (13, 41365, 39, 0.0, 2.0, 0, 0),     # few rows, many tokens: narrow tiles, dh in many splits
    (100, 30000, 75, 0.4, 2.0, 2, 1),
    (600, 700, 300, 0.2, 2.0, 1, 1),
    (20000, 50, 16, 0.3, 2.0, 0, 0),     # many rows, few tokens
    (7, 900, 150, 0.0, 2.0, 4, 2),       # dW's rows start on 4 bytes
])
def test_loss_and_gradients(handle, rows, V, d, ignored, gain, pad, offset):
    h, w, t, gl = _inputs(rows, V, d, rows + V + d, gain, ignored, extra=8 if pad else 0)
    ce = handle(V, d, rows)
    loss, lse = _loss(ce, h, w, t)
    dh, dw = _grad(ce, h, w, t, lse, gl, pad, offset)
    assert fr.fr_ce_status(ce) == fr.FR_OK
    ref = _reference(h, w, t, gl)
    _close(lse, ref["lse"])
    _close(loss, ref["loss"])
    _close(dh, ref["dh"])
    _close(dw, ref["dw"])
    # the same again, bit for bit, and each gradient alone
    a, b = _grad(ce, h, w, t, lse, gl, pad, offset)
    assert torch.equal(a, dh) and torch.equal(b, dw)
    a, b = torch.empty_like(dh), torch.empty_like(dw)
    fr.fr_ce_grad(ce, h, w, t, lse, gl, a, None)
    fr.fr_ce_grad(ce, h, w, t, lse, gl, None, b)
    assert torch.equal(a, dh) and torch.equal(b, dw)


def test_gradients_against_differences(handle):
    """The loss along a direction: (L(h + e) - L(h - e)) / 2 in double, from
    losses of bf16 inputs moved by one exact step, against the gradients.  The
    central difference is off by a third derivative (|x| moved by at most
    2^-4: under 2^-12 of the magnitude sum) and each gradient by its bound."""
    rows, V, d = 40, 90, 24
    h, w, t, gl = _inputs(rows, V, d, 3)
    ce = handle(V, d, rows)
    loss, lse = _loss(ce, h, w, t)
    dh, dw = _grad(ce, h, w, t, lse, gl)
    ref = _reference(h, w, t, gl)

    def total(hh, ww):
        x = hh @ ww.T
        live = t.cpu() >= 0
        each = torch.logsumexp(x, 1) - x.gather(1, t.long().cpu().clamp(min=0)[:, None])[:, 0]
        return (each * gl.double().cpu())[live].sum()

    hd, wd = h.double().cpu(), w.double().cpu()
    e = 2.0 ** -10
    g = torch.Generator().manual_seed(1)
    for _ in range(4):
        sh, sw = torch.randn(rows, d, generator=g).double().sign(), torch.randn(V, d, generator=g).double().sign()
        diff = (total(hd + e * sh, wd + e * sw) - total(hd - e * sh, wd - e * sw)) / (2 * e)
        along = (dh.double().cpu() * sh).sum() + (dw.double().cpu() * sw).sum()
        slack = ref["dh"][1].sum() + ref["dw"][1].sum()
        third = 2.0 ** -12 * gl.double().abs().sum().cpu()
        assert abs(diff - along) <= slack + third


@pytest.mark.parametrize("scale", [1e-36, 1e-41, 1e34])
def test_small_and_large_incoming_gradients(handle, scale):
    """Gradients of tiny (normal and subnormal) and huge incoming values: bf16
    has fp32's exponent range, so they are those of 1 times the scale; a result
    below 2^-126 is off by at most a subnormal step of bf16 (2^-133)."""
    rows, V, d = 50, 120, 32
    h, w, t, gl = _inputs(rows, V, d, 13, ignored=0.1)
    gl = (gl.sign() * scale).contiguous()  # one magnitude
    ce = handle(V, d, rows)
    loss, lse = _loss(ce, h, w, t)
    dh, dw = _grad(ce, h, w, t, lse, gl)
    ref = _reference(h, w, t, gl)
    for got, name in ((dh, "dh"), (dw, "dw")):
        want, bound = ref[name]
        # fp32 products and sums below 2^-126 lose up to half a subnormal step each
        slack = 2.0 ** -133 + (rows + V) * 2.0 ** -149
        assert torch.all((got.double().cpu() - want).abs() <= bound + slack)


def test_no_incoming_gradient(handle):
    rows, V, d = 30, 70, 16
    h, w, t, gl = _inputs(rows, V, d, 14)
    ce = handle(V, d, rows)
    loss, lse = _loss(ce, h, w, t)
    dh, dw = _grad(ce, h, w, t, lse, torch.zeros_like(gl))
    assert torch.all(dh == 0) and torch.all(dw == 0)


def test_a_nan_in_one_row_stays_in_its_gradients(handle):
    """A NaN or infinite incoming gradient of one row reaches that row's dh and,
    as the formula says, dW; the other rows' dh are what they were."""
    rows, V, d = 40, 90, 24
    h, w, t, gl = _inputs(rows, V, d, 15, ignored=0.0)
    ce = handle(V, d, rows)
    loss, lse = _loss(ce, h, w, t)
    ref = _reference(h, w, t, gl)
    for bad in (float("nan"), float("inf")):
        g2 = gl.clone()
        g2[7] = bad
        dh, dw = _grad(ce, h, w, t, lse, g2)
        keep = [r for r in range(rows) if r != 7]
        _close(dh[keep], tuple(x[keep] for x in ref["dh"]))
        assert not torch.any(torch.isfinite(dh[7])) and not torch.all(torch.isfinite(dw))


def test_rows_that_do_not_count_reach_nothing(handle):
    rows, V, d = 200, 500, 64
    h, w, t, gl = _inputs(rows, V, d, 11, ignored=0.4)
    ref = _reference(h, w, t, gl)
    dead = t < 0
    h[dead] = float("nan")
    h[int(torch.nonzero(dead)[0, 0])] = float("inf")
    gl[dead] = float("nan")
    ce = handle(V, d, rows)
    loss, lse = _loss(ce, h, w, t)
    dh, dw = _grad(ce, h, w, t, lse, gl)
    assert fr.fr_ce_status(ce) == fr.FR_OK
    for got, name in ((loss, "loss"), (lse, "lse"), (dh, "dh"), (dw, "dw")):
        _close(got, ref[name])
    assert torch.all(loss[dead] == 0) and torch.all(lse[dead] == 0) and torch.all(dh[dead] == 0)


@pytest.mark.parametrize("rows", [0, 1, 150])
def test_no_row_counts(handle, rows):
    V, d = 300, 40
    h, w, t, gl = _inputs(rows, V, d, 1, ignored=2.0)
    ce = handle(V, d, 150)
    h.fill_(float("nan"))
    loss, lse = _loss(ce, h, w, t)
    dh, dw = _grad(ce, h, w, t, lse, gl)
    assert fr.fr_ce_status(ce) == fr.FR_OK
    for x in (loss, lse, dh, dw):
        assert torch.all(x == 0)


def test_fewer_rows_than_the_handle_holds(handle):
    V, d = 9000, 96
    h, w, t, gl = _inputs(400, V, d, 21)
    ce = handle(V, d, 20000)  # sized for far more: pieces and tiles go by the call's rows
    for n in (400, 3, 129):
        loss, lse = _loss(ce, h[:n], w, t[:n])
        dh, dw = _grad(ce, h[:n], w, t[:n], lse, gl[:n])
        ref = _reference(h[:n], w, t[:n], gl[:n])
        for got, name in ((loss, "loss"), (lse, "lse"), (dh, "dh"), (dw, "dw")):
            _close(got, ref[name])


def test_targets_out_of_range_are_recorded(handle):
    h, w, t, gl = _inputs(6, 50, 16, 2, ignored=0.0)
    ref = _reference(h, w, torch.where(torch.arange(6).cuda() % 3 == 1, -1, t).int(), gl)
    t[1], t[4] = 50, -2
    ce = handle(50, 16, 6)
    loss, lse = _loss(ce, h, w, t)
    assert fr.fr_ce_status(ce) == fr.FR_ERR_CODE_RANGE
    fr.fr_ce_clear_status(ce)
    assert fr.fr_ce_status(ce) == fr.FR_OK
    assert torch.all(torch.isnan(loss[[1, 4]])) and torch.all(torch.isnan(lse[[1, 4]]))
    keep = [0, 2, 3, 5]
    _close(loss[keep], tuple(x[keep] for x in ref["loss"]))
    dh, dw = _grad(ce, h, w, t, lse, gl)
    assert fr.fr_ce_status(ce) == fr.FR_ERR_CODE_RANGE
    _close(dh, ref["dh"])
    _close(dw, ref["dw"])


def test_a_row_that_is_not_finite_is_recorded(handle):
    h, w, t, gl = _inputs(5, 40, 16, 4, ignored=0.0)
    h[3, 2] = float("nan")
    ce = handle(40, 16, 5)
    loss, lse = _loss(ce, h, w, t)
    assert fr.fr_ce_status(ce) == fr.FR_ERR_NAN_LOGIT
    assert torch.isnan(loss[3]) and torch.all(torch.isfinite(loss[[0, 1, 2, 4]]))


def test_graph_and_another_stream(handle):
    rows, V, d = 150, 9000, 72
    sets = [_inputs(rows, V, d, s, ignored=i) for s, i in ((1, 0.1), (2, 0.7))]
    ce = handle(V, d, rows)
    want = []
    for h, w, t, gl in sets:
        loss, lse = _loss(ce, h, w, t)
        want.append((loss, *_grad(ce, h, w, t, lse, gl)))
    h, w, t, gl = (x.clone(memory_format=torch.preserve_format) for x in sets[0])
    h, w = _padded(rows, d), _padded(V, d)
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    dh, dw = torch.empty(rows, d, dtype=BF16, device="cuda"), torch.empty(V, d, dtype=BF16, device="cuda")

    def run():
        fr.fr_ce_loss(ce, h, w, t, loss, lse)
        fr.fr_ce_grad(ce, h, w, t, lse, gl, dh, dw)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        run()
    for (a, b, c, e), (x, y, z) in list(zip(sets, want)) * 2:  # the number of rows that count changes between replays
        h.copy_(a), w.copy_(b), t.copy_(c), gl.copy_(e)
        graph.replay()
        assert torch.equal(loss, x) and torch.equal(dh, y) and torch.equal(dw, z)
    with torch.cuda.stream(s):
        s.wait_stream(torch.cuda.default_stream())
        dw.fill_(4.0)
        run()
    s.synchronize()
    assert torch.equal(dw, want[1][2])


def test_a_wait_that_expires(handle):
    """The producer issues no copies: loss and gradient give up after 1 ms,
    record it, and the handle works again afterwards."""
    h, w, t, gl = _inputs(60, 700, 64, 8)
    ref = _reference(h, w, t, gl)
    ce = handle(700, 64, 60)
    loss, lse = _loss(ce, h, w, t)
    dh, dw = torch.empty(60, 64, dtype=BF16, device="cuda"), torch.empty(700, 64, dtype=BF16, device="cuda")
    for call in (lambda: fr.fr_ce_loss(ce, h, w, t, loss.clone(), lse.clone()),
                 lambda: fr.fr_ce_grad(ce, h, w, t, lse, gl, dh, dw)):
        fr.fr_ce_set_wait_test(ce, 1_000_000, True)
        call()
        assert fr.fr_ce_status(ce) == fr.FR_ERR_DEVICE
        fr.fr_ce_set_wait_test(ce, 0, False)
        fr.fr_ce_clear_status(ce)
    dh, dw = _grad(ce, h, w, t, lse, gl)
    assert fr.fr_ce_status(ce) == fr.FR_OK
    _close(dh, ref["dh"])
    _close(dw, ref["dw"])


def test_refusals(handle):
    h, w, t, gl = _inputs(8, 40, 32, 0)
    ce = handle(40, 32, 8)
    loss, lse = torch.empty(8, device="cuda"), torch.empty(8, device="cuda")
    dh, dw = torch.empty(8, 32, dtype=BF16, device="cuda"), torch.empty(40, 32, dtype=BF16, device="cuda")
    for bad in (lambda: fr.fr_ce_loss(ce, h.float(), w, t, loss, lse), lambda: fr.fr_ce_loss(ce, h[:, :31], w, t, loss, lse),
                lambda: fr.fr_ce_loss(ce, h, w[:39], t, loss, lse), lambda: fr.fr_ce_loss(ce, h, w, t.long(), loss, lse),
                lambda: fr.fr_ce_loss(ce, h, w, t, loss[:7], lse), lambda: fr.fr_ce_loss(ce, h, w, t.cpu(), loss, lse),
                lambda: fr.fr_ce_grad(ce, h, w, t, lse, gl[:7], dh, dw), lambda: fr.fr_ce_grad(ce, h, w, t, lse, gl, dh.float(), dw),
                lambda: fr.fr_ce_grad(ce, h, w, t, lse, gl, dh, dw[:39])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(fr.FrError):  # neither gradient
        fr.fr_ce_grad(ce, h, w, t, lse, gl, None, None)
    with pytest.raises(fr.FrError):  # more rows than the handle holds
        fr.fr_ce_loss(ce, *_inputs(9, 40, 32, 0)[:3], torch.empty(9, device="cuda"), torch.empty(9, device="cuda"))
    odd = torch.zeros(8, 33, dtype=BF16, device="cuda")[:, :32]
    with pytest.raises(fr.FrError):  # pitch not a multiple of 8
        fr.fr_ce_loss(ce, odd, w, t, loss, lse)
    with pytest.raises(fr.FrError):  # base not on 16 bytes
        fr.fr_ce_loss(ce, torch.zeros(8 * 32 + 8, dtype=BF16, device="cuda")[1:257].view(8, 32), w, t, loss, lse)


@pytest.mark.parametrize("big,small", [(1e30, 1e-10), (1e10, 1e-33), (3e38, 1e-12), (1.5, 1e-30), (2.0 ** 64, 2.0 ** -60)])
def test_incoming_gradients_of_very_different_sizes(handle, big, small):
    """A row's dh does not depend on the other rows' incoming gradients: rows
    of small ones beside rows of large ones have the same relative bounds.  Only
    entries of G that lie below 2^-126 at the scale they are kept at lose to subnormals."""
    rows, V, d = 60, 130, 40
    h, w, t, gl = _inputs(rows, V, d, 17, gain=1.0, ignored=0.1)
    w *= 0.125  # results of the largest incoming gradients stay finite
    gl = torch.where(torch.arange(rows, device="cuda") % 2 == 0, big, small) * torch.where(gl < 0, -0.5, 1.0)
    gl = gl.float().contiguous()
    ce = handle(V, d, rows)
    loss, lse = _loss(ce, h, w, t)
    dh, dw = _grad(ce, h, w, t, lse, gl)
    ref = _reference(h, w, t, gl)
    # subnormal steps: of G (2^-134, half of bf16's) in a sum over V and of the sums, at
    # the scale that G is kept at (below 2, or the largest incoming gradient over 2^64)
    slack = (V * 2.0 ** -134 * float(w.abs().max()) + (rows + V) * 2.0 ** -149) * max(2.0, big * 2.0 ** -64) + 2.0 ** -134
    _close(dh, (ref["dh"][0], ref["dh"][1] + slack))
    if big < 1e38:  # (dW sums many rows)
        slack *= max(1.0, float(h.abs().max()) / float(w.abs().max()))
        _close(dw, (ref["dw"][0], ref["dw"][1] + slack))


@pytest.mark.parametrize("V,d,rows", [(5120, 256, 1), (151936, 2048, 96), (300, 40, 150), (151936, 64, 2048), (9000, 96, 40000)])
def test_a_handle_takes_the_memory_that_the_header_states(handle, V, d, rows):
    """Of include/fr.h's account for fr_ce_init, and of no more: each of six
    allocations is rounded up to the driver's 2 MB."""
    handle(64, 64, 1)  # (what the first init loads)
    torch.cuda.synchronize()
    before = torch.cuda.mem_get_info()[0]
    handle(V, d, rows)
    taken = before - torch.cuda.mem_get_info()[0]
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    R, W, D = -(-rows // 256) * 256, -(-V // 256) * 256, -(-d // 8) * 8
    piece = max(512 << 20, 8192 * R)
    stated = R * (2 * D + W / 16 + 20) + (1 << 19) + 4 * D * max(R, 512 * sms // -(-d // 256))
    stated += 2 * W * R if 2 * W * R <= piece else 2 * piece
    assert 0 < taken <= stated + 6 * (2 << 20)


def _spread(t, borders):
    """Targets of the counted rows dealt over the ranges between `borders`, first and last token of each among them."""
    live = torch.nonzero(t >= 0)[:, 0]
    at = []
    for lo, hi in zip(borders, borders[1:]):
        at += [lo, hi - 1, (lo + hi) // 2]
    t[live] = torch.tensor(at, dtype=torch.int32, device="cuda").repeat(len(live) // len(at) + 1)[:len(live)]


@pytest.mark.parametrize("rows,V,d,counted,pieces", [
    (66000, 8500, 40, 0.01, (0, 4096, 8192, 8500)),           # three pieces of G, few of many rows count
    (66000, 8200, 264, 0.005, (0, 4096, 8192, 8200)),         # a last piece of 8 tokens, two column tiles of dh
    (200, 1048876, 8, 0.08, (0, 1048576, 1048876)),           # pairs: dh in splits, most of them empty in the last piece
    (100, 1048876, 8, 0.15, (0, 1048576, 1048876)),           # the same on single CTAs
])
def test_gradients_over_several_pieces_of_the_vocabulary(handle, rows, V, d, counted, pieces):
    """G is kept for 512 MB of a handle's rows by tokens at a time (4,096 tokens at
    least).  The targets lie in every piece, so that a piece that was lost or added
    twice would be off by a whole row of W or h.  An fp32 chain of dh has at most
    16,384 terms (a split of a piece), and the splits and pieces are added to it."""
    h, w, t, gl = _inputs(rows, V, d, rows + V, ignored=1 - counted, extra=8)
    _spread(t, pieces)
    ce = handle(V, d, rows)
    loss, lse = _loss(ce, h, w, t)
    dh, dw = _grad(ce, h, w, t, lse, gl, 3, 1)
    assert fr.fr_ce_status(ce) == fr.FR_OK
    live = t >= 0
    assert torch.all(dh[~live] == 0)
    ref = _reference(h[live], w, t[live], gl[live])
    want, bound = ref["dh"]
    if V > 16384:
        hd, wd, at = h[live].double().cpu(), w.double().cpu(), t[live].long().cpu()[:, None]
        G = torch.softmax(hd @ wd.T, 1)
        G = (G - torch.zeros_like(G).scatter_(1, at, 1.0)) * gl[live].double().cpu()[:, None]
        bound = bound - (V - 16384 - 512) * 2.0 ** -23 * (G.abs() @ wd.abs())
    _close(dh[live], (want, bound))
    _close(dw, ref["dw"])
    _close(loss[live], ref["loss"])
    a, b = _grad(ce, h, w, t, lse, gl, 3, 1)
    assert torch.equal(a, dh) and torch.equal(b, dw)
    a, b = torch.empty_like(dh), torch.empty_like(dw)
    fr.fr_ce_grad(ce, h, w, t, lse, gl, a, None)
    fr.fr_ce_grad(ce, h, w, t, lse, gl, None, b)
    assert torch.equal(a, dh) and torch.equal(b, dw)


@pytest.mark.parametrize("V", [700, 1300])
def test_more_rows_than_a_group_of_tiles_holds(handle, V):
    """Tile rows are walked 32 (8,192 rows) at a time: counted rows beyond, by several column tiles."""
    rows, d = 9100, 24
    h, w, t, gl = _inputs(rows, V, d, V, ignored=0.02)
    ce = handle(V, d, rows)
    loss, lse = _loss(ce, h, w, t)
    dh, dw = _grad(ce, h, w, t, lse, gl)
    ref = _reference(h, w, t, gl)
    for got, name in ((loss, "loss"), (lse, "lse"), (dh, "dh"), (dw, "dw")):
        _close(got, ref[name])
