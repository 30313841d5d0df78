"""Token embedding and its gradient vs the formulas in double.

Tolerances, from the arithmetic: the lookup is one fp32 product and one
rounding to the output type, which torch's float32 product and conversion do
too, so it is compared bit for bit.  A gradient is an fp32 sum of m terms in
some order (error at most m * 2^-24 * sum |g|), one product by the scale, one
addition, and one rounding of the result to the table's type (half a step)."""
import numpy as np
import pytest
import torch

from trie_constrained_beam_fr_b200 import fr

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def _half_step(dtype):
    return torch.finfo(dtype).eps / 2


def _rand(g, rows, cols, dtype, pad=0, offset=0):
    """A [rows, cols] CUDA tensor whose rows are `pad` elements further apart
    and start `offset` elements into their storage."""
    flat = torch.full((rows * (cols + pad) + offset + 8,), 7.0, dtype=dtype, device="cuda")
    t = flat[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    t.copy_(torch.randn(rows, cols, generator=g))
    return t


def _tokens(g, n, V, kind):
    if kind == "same":
        t = torch.full((n,), V - 1)
    elif kind == "dead":
        t = torch.full((n,), -1)
    elif kind == "hot":
        t = (torch.rand(n, generator=g) ** 4 * V).long().clamp(max=V - 1)
        t[torch.rand(n, generator=g) < 0.2] = -1
    else:
        t = torch.randint(0, V, (n,), generator=g)
    return t.int()


@pytest.fixture
def handle():
    made = []

    def make(V, d, n):
        made.append(fr.fr_embed_init(V, d, n))
        return made[-1]

    yield make
    for h in made:
        fr.fr_embed_destroy(h)


@pytest.mark.parametrize("tin", [F32, BF16])
@pytest.mark.parametrize("tout", [F32, BF16])
@pytest.mark.parametrize("n,V,d,pad,offset", [
    (1, 1, 1, 0, 0), (7, 33, 8, 0, 0), (100, 50, 129, 0, 0), (64, 1000, 2048, 0, 0), (65, 70, 24, 8, 8), (30, 70, 24, 3, 1),
])
def test_lookup(handle, tin, tout, n, V, d, pad, offset):
    g = torch.Generator().manual_seed(n + d)
    table = _rand(g, V, d, tin, pad, offset)
    out = _rand(g, n, d, tout, pad, offset)
    whole = out._base.clone()
    tok = _tokens(g, n, V, "hot").cuda()
    h = handle(V, d, n)
    fr.fr_embed_lookup(h, table, tok, out, scale=1.7)
    assert fr.fr_embed_status(h) == fr.FR_OK
    want = torch.where((tok >= 0)[:, None], table[tok.clamp(min=0).long()].float() * np.float32(1.7), 0.0).to(tout)
    assert torch.equal(out, want)
    # nothing between or behind the rows was written
    mask = torch.ones_like(whole, dtype=torch.bool)
    mask[offset:offset + n * (d + pad)].view(n, d + pad)[:, :d] = False
    assert torch.equal(out._base[mask], whole[mask])


def _grad_reference(grad, tok, V, scale, before):
    g, t = grad.double().cpu(), tok.long().cpu()
    live = t >= 0
    total, mag, count = (torch.zeros(V, grad.shape[1], dtype=torch.float64) for _ in range(3))
    total.index_add_(0, t[live], g[live])
    mag.index_add_(0, t[live], g[live].abs())
    count.index_add_(0, t[live], torch.ones_like(g[live]))
    want = total * scale + (0 if before is None else before.double().cpu())
    bound = (count + 2) * 2.0 ** -24 * mag * abs(scale) + (0 if before is None else 2.0 ** -24 * before.double().abs().cpu())
    return want, bound


@pytest.mark.parametrize("kind", ["any", "hot", "same", "dead"])
@pytest.mark.parametrize("n,V,d,tg,tt,add,pad,offset", [
    (1, 1, 1, F32, F32, False, 0, 0),
    (31, 40, 16, BF16, BF16, True, 0, 0),
    (33, 1000, 129, F32, F32, True, 0, 0),
    (1000, 77, 64, BF16, F32, False, 0, 0),
    (2049, 5000, 40, F32, BF16, False, 8, 8),
    (4100, 300000, 24, BF16, BF16, True, 5, 3),   # 19 bits of tokens: three sort passes
    (9000, 64, 136, BF16, BF16, False, 0, 0),     # runs over many chunks
    (1024, 500, 264, F32, BF16, False, 0, 0),
    (1025, 500, 264, F32, BF16, False, 0, 0),
    (2048, 500, 264, F32, BF16, False, 0, 0),     # the most tokens of the one-kernel form
    (2049, 500, 264, F32, BF16, False, 0, 0),     # the fewest of the sorted form
    (2047, 300, 401, F32, BF16, True, 1, 1),
    (600, 40, 12000, BF16, F32, True, 0, 0),      # few tokens, sorted: long rows
    (300000, 700, 8, F32, F32, False, 0, 0),      # several tiles per sorting CTA
    (32769, 300001, 9, F32, F32, False, 0, 0),
    (20000, 511, 16, F32, F32, False, 0, 0),      # keys that fill their digits
    (5000, 262143, 16, F32, F32, False, 0, 0),
])
def test_grad(handle, kind, n, V, d, tg, tt, add, pad, offset):
    g = torch.Generator().manual_seed(n + V)
    grad = _rand(g, n, d, tg, pad, offset)
    table = _rand(g, V, d, tt, pad, offset)
    whole, before = table._base.clone(), table.clone()
    tok = _tokens(g, n, V, kind).cuda()
    h = handle(V, d, n)
    fr.fr_embed_grad(h, grad, tok, table, scale=0.3, accumulate=add)
    assert fr.fr_embed_status(h) == fr.FR_OK
    scale = float(np.float32(0.3))
    want, bound = _grad_reference(grad, tok, V, scale, before if add else None)
    got = table.double().cpu()
    assert torch.all((got - want).abs() <= bound + _half_step(tt) * (want.abs() + bound))
    untouched = torch.ones(V, dtype=torch.bool)
    untouched[tok[tok >= 0].long().cpu()] = False
    if add:
        assert torch.equal(table.cpu()[untouched], before.cpu()[untouched])
    else:
        assert torch.all(got[untouched] == 0)
    mask = torch.ones_like(whole, dtype=torch.bool)
    mask[offset:offset + V * (d + pad)].view(V, d + pad)[:, :d] = False
    assert torch.equal(table._base[mask], whole[mask])
    first = table.clone()  # the same order of sums again
    table.copy_(before)
    fr.fr_embed_grad(h, grad, tok, table, scale=0.3, accumulate=add)
    assert torch.equal(table, first)


@pytest.mark.parametrize("runs", [
    (1024, 1024, 1, 1023, 1025, 2048), (1000, 24, 1024, 1025, 31, 33, 960, 3000), (32, 992, 32, 32, 1000, 1), (1040, 1000, 40, 2000, 16, 40, 8),
    (33000, 500, 33300, 7),
])
@pytest.mark.parametrize("d", [8, 70, 520])
def test_grad_of_runs_at_the_joins_borders(handle, runs, d):
    """Tokens repeated so often that their sums are put together from many
    pieces, beginning and ending on, before and behind the pieces' borders."""
    g = torch.Generator().manual_seed(sum(runs) + d)
    n, V = sum(runs), len(runs) + 2
    tok = torch.repeat_interleave(torch.arange(len(runs)), torch.tensor(runs))[torch.randperm(n, generator=g)].int().cuda()
    grad, table = torch.randn(n, d, generator=g).to(BF16).cuda(), torch.full((V, d), 3.0, device="cuda")
    h = handle(V, d, n)
    fr.fr_embed_grad(h, grad, tok, table)
    want, bound = _grad_reference(grad, tok, V, 1.0, None)
    assert torch.all((table.double().cpu() - want).abs() <= bound + _half_step(F32) * (want.abs() + bound))
    first = table.clone()
    fr.fr_embed_grad(h, grad, tok, table)
    assert torch.equal(table, first)


def test_grad_is_the_lookups_gradient(handle):
    """sum(grad * lookup(T + e E)) differs from sum(grad * lookup(T)) by
    e * sum(dT * E): the lookup is linear, so the difference is exact up to
    fp32 rounding (64-bit sums of fp32 lookups, values of order 1)."""
    g = torch.Generator().manual_seed(5)
    n, V, d = 500, 60, 33
    table, E, grad = _rand(g, V, d, F32), _rand(g, V, d, F32), _rand(g, n, d, F32)
    tok = _tokens(g, n, V, "hot").cuda()
    h = handle(V, d, n)
    a, b, dT = torch.empty(n, d, device="cuda"), torch.empty(n, d, device="cuda"), torch.empty(V, d, device="cuda")
    moved = (table + 0.5 * E).contiguous()
    fr.fr_embed_lookup(h, table, tok, a, scale=2.0)
    fr.fr_embed_lookup(h, moved, tok, b, scale=2.0)
    fr.fr_embed_grad(h, grad, tok, dT, scale=2.0)
    left = ((b.double() - a.double()) * grad.double()).sum().item()
    right = (dT.double() * (moved.double() - table.double())).sum().item()
    mag = (grad.double().abs().sum() * 4.0 * (table.abs().max() + E.abs().max()).double()).item()
    assert abs(left - right) <= mag * 2.0 ** -22


def test_fewer_tokens_and_none(handle):
    g = torch.Generator().manual_seed(9)
    table, out = _rand(g, 20, 16, F32), _rand(g, 10, 16, F32)
    h = handle(20, 16, 10)
    tok = _tokens(g, 10, 20, "any").cuda()
    before = out.clone()
    fr.fr_embed_lookup(h, table, tok[:3], out[:3])
    assert torch.equal(out[3:], before[3:]) and torch.equal(out[:3], table[tok[:3].long()])
    fr.fr_embed_lookup(h, table, tok[:0], out[:0])
    fr.fr_embed_grad(h, out[:0], tok[:0], table)  # no tokens: zeros everywhere
    assert torch.all(table == 0)
    table.fill_(3.0)
    fr.fr_embed_grad(h, out[:0], tok[:0], table, accumulate=True)
    assert torch.all(table == 3)


def test_tokens_out_of_range_are_recorded(handle):
    h = handle(8, 16, 4)
    table, out = torch.ones(8, 16, device="cuda"), torch.full((4, 16), 9.0, device="cuda")
    tok = torch.tensor([0, 8, -2, 7], dtype=torch.int32, device="cuda")
    fr.fr_embed_lookup(h, table, tok, out)
    assert fr.fr_embed_status(h) == fr.FR_ERR_CODE_RANGE
    assert out[:, 0].tolist() == [1.0, 0.0, 0.0, 1.0]
    fr.fr_embed_clear_status(h)
    assert fr.fr_embed_status(h) == fr.FR_OK
    fr.fr_embed_grad(h, out, tok, table)
    assert fr.fr_embed_status(h) == fr.FR_ERR_CODE_RANGE
    assert table[:, 0].tolist() == [1.0, 0, 0, 0, 0, 0, 0, 1.0]


def test_nan_of_a_dead_token_reaches_nothing(handle):
    h = handle(6, 8, 3)
    grad = torch.ones(3, 8, device="cuda")
    grad[1] = float("nan")
    tok = torch.tensor([2, -1, 2], dtype=torch.int32, device="cuda")
    table = torch.empty(6, 8, device="cuda")
    fr.fr_embed_grad(h, grad, tok, table)
    assert table[:, 0].tolist() == [0, 0, 2, 0, 0, 0]


def test_another_stream_and_a_graph(handle):
    g = torch.Generator().manual_seed(2)
    n, V, d = 300, 90, 64
    h = handle(V, d, n)
    table, grad = _rand(g, V, d, BF16), _rand(g, n, d, BF16)
    toks = [_tokens(g, n, V, k).cuda() for k in ("any", "hot")]
    want = []
    for t in toks:
        out, dT = torch.empty(n, d, dtype=BF16, device="cuda"), torch.empty(V, d, dtype=BF16, device="cuda")
        fr.fr_embed_lookup(h, table, t, out)
        fr.fr_embed_grad(h, grad, t, dT)
        want.append((out, dT))
    out, dT, tok = torch.empty_like(want[0][0]), torch.empty_like(want[0][1]), toks[0].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        fr.fr_embed_lookup(h, table, tok, out)
        fr.fr_embed_grad(h, grad, tok, dT)
    for t, (o, dt) in list(zip(toks, want)) * 2:
        tok.copy_(t)
        out.fill_(5), dT.fill_(5)
        graph.replay()
        assert torch.equal(out, o) and torch.equal(dT, dt)
    with torch.cuda.stream(s):
        s.wait_stream(torch.cuda.default_stream())
        out.fill_(5)
        fr.fr_embed_lookup(h, table, toks[1], out)
    s.synchronize()
    assert torch.equal(out, want[1][0])


def test_refusals(handle):
    h = handle(8, 16, 4)
    table, out, tok = torch.ones(8, 16, device="cuda"), torch.ones(4, 16, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad in (lambda: fr.fr_embed_lookup(h, table[:7], tok, out), lambda: fr.fr_embed_lookup(h, table, tok.long(), out),
                lambda: fr.fr_embed_lookup(h, table, tok, out[:3]), lambda: fr.fr_embed_lookup(h, table.half(), tok, out),
                lambda: fr.fr_embed_lookup(h, table.cpu(), tok, out), lambda: fr.fr_embed_lookup(h, table, tok, out[:1].expand(4, 16)),
                lambda: fr.fr_embed_lookup(h, table.t().contiguous().t(), tok, out),
                lambda: fr.fr_embed_grad(h, out, tok, table[:, :15])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(fr.FrError):
        fr.fr_embed_lookup(h, table, torch.zeros(5, dtype=torch.int32, device="cuda"), torch.ones(5, 16, device="cuda"))


@pytest.mark.parametrize("n,d", [(1400, 2048), (1700, 1536), (2048, 1280), (1000, 2056)])
def test_the_sums_order_does_not_depend_on_where_rows_start(handle, n, d):
    """The same tokens and values in rows that start on 16 bytes and in rows that
    start anywhere: the same sums, bit for bit."""
    g = torch.Generator().manual_seed(n + d)
    V = 40
    tok = _tokens(g, n, V, "hot").cuda()
    grad = _rand(g, n, d, F32)
    h = handle(V, d, n)
    got = []
    for pad, offset in ((0, 0), (1, 0), (3, 1)):
        src, table = _rand(g, n, d, F32, pad, offset), _rand(g, V, d, F32, pad, offset)
        src.copy_(grad)
        fr.fr_embed_grad(h, src, tok, table, scale=0.3)
        got.append(table.clone())
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])
