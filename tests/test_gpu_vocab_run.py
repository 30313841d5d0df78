"""The vocabulary operators as a program uses them together: a training step of
a model whose embedding and lm_head share one table, and a decode whose steps
embed the beams' tokens and project them through an 8-bit lm_head."""
import pytest
import torch

from trie_constrained_beam_fr_b200 import fr, synth

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def test_a_training_step_with_a_tied_table():
    """embedding -> two linear layers with a tanh -> cross entropy over the same
    table; the table's gradient is the sum of both ends.  Against the same
    network in double (from the bf16 values that the kernels see); the network
    between rounds its activations to bf16, so the check is on norms: each
    rounding is half a step (2^-8) of its tensor, and six tensors are rounded
    on the way (embedding, hidden, G, its two gradients, the table's gradient
    twice): 8 * 2^-8 of the norm."""
    torch.manual_seed(0)
    n, V, d = 333, 777, 96
    table = (torch.randn(V, d, device="cuda") / d ** 0.5).to(BF16)
    w1 = (torch.randn(d, d, device="cuda") / d ** 0.5).to(BF16).float()
    tokens = torch.randint(0, V, (n,), device="cuda", dtype=torch.int32)
    targets = torch.randint(0, V, (n,), device="cuda", dtype=torch.int32)
    tokens[::17] = -1
    targets[::5] = -1
    scale = d ** 0.5
    counted = int((targets >= 0).sum())

    em, ce = fr.fr_embed_init(V, d, n), fr.fr_ce_init(V, d, n)
    try:
        x = torch.empty(n, d, dtype=BF16, device="cuda")
        fr.fr_embed_lookup(em, table, tokens, x, scale)
        x1 = x.float().requires_grad_(True)
        hidden_f = torch.tanh(x1 @ w1)
        hidden = hidden_f.detach().to(BF16)
        loss, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
        fr.fr_ce_loss(ce, hidden, table, targets, loss, lse)
        gl = torch.full((n,), 1.0 / counted, device="cuda")
        dh, dT = torch.empty_like(hidden), torch.empty_like(table)
        fr.fr_ce_grad(ce, hidden, table, targets, lse, gl, dh, dT)
        hidden_f.backward(dh.float())
        fr.fr_embed_grad(em, x1.grad, tokens, dT, scale, accumulate=True)
        assert fr.fr_embed_status(em) == fr.FR_OK and fr.fr_ce_status(ce) == fr.FR_OK
    finally:
        fr.fr_embed_destroy(em)
        fr.fr_ce_destroy(ce)

    T = table.double().cpu().requires_grad_(True)
    tok, tgt = tokens.long().cpu(), targets.long().cpu()
    xr = torch.where((tok >= 0)[:, None], T[tok.clamp(min=0)] * scale, torch.zeros((), dtype=torch.float64))
    hr = torch.tanh(xr @ w1.double().cpu())
    want = torch.nn.functional.cross_entropy((hr @ T.T)[tgt >= 0], tgt[tgt >= 0])
    want.backward()
    got = loss.double().sum().item() / counted
    # the loss moves by at most the largest change of a logit: |h| is rounded by
    # 2^-8 twice (embedding, hidden), and the logits are of order |h| |T|
    logit = (hr.detach().norm(dim=1).max() * T.detach().norm(dim=1).max()).item()
    assert abs(got - want.item()) <= 4 * 2.0 ** -8 * logit
    err = (dT.double().cpu() - T.grad).norm() / T.grad.norm()
    assert err <= 8 * 2.0 ** -8


def test_a_decode_through_the_8_bit_lm_head():
    """Beam steps from fr_i8_matmul's logits and from fr_i8_lse's rows agree,
    and the survivors' scores are the sums of their tokens' log-probabilities
    in double (each log-probability is off by at most a few 1e-6: 3 steps of
    fp32, logits of order 10)."""
    w = synth.scaled(synth.WORKLOADS["tiny"], B=3)
    sids = synth.workload_catalog(w)
    B, K, V, D, d = w.B, w.K, w.V, w.depth, 80
    g = torch.Generator().manual_seed(3)
    table = torch.randn(V, d, generator=g).cuda()
    root = torch.randn(B, d, generator=g).cuda()
    wq, ws = torch.empty(V, d, dtype=torch.int8, device="cuda"), torch.empty(V, device="cuda")
    fr.fr_i8_quantize(torch.randn(V, d, generator=g).cuda(), wq, ws)
    span = sum(w.codebook_sizes)
    trie = fr.fr_trie_build(torch.from_numpy(sids).cuda(), w.codebook_sizes, w.sid_base)
    beams = [fr.fr_beam_init(trie, B, K, V, "f32") for _ in range(2)]
    em = fr.fr_embed_init(V, d, B * K)
    i8 = fr.fr_i8_init(wq, ws, B * K, w.sid_base, span)
    try:
        hidden = torch.zeros(B, K, d, device="cuda")
        hidden[:, 0] = root
        q, s = torch.empty(B * K, d, dtype=torch.int8, device="cuda"), torch.empty(B * K, device="cuda")
        logits, lse, sl = torch.empty(B, K, V, device="cuda"), torch.empty(B * K, device="cuda"), torch.empty(B * K, span, device="cuda")
        scores = torch.zeros(B, K, dtype=torch.float64)
        for t in range(D):
            fr.fr_i8_quantize(hidden.view(B * K, d), q, s)
            fr.fr_i8_matmul(i8, q, s, logits.view(B * K, V))
            fr.fr_i8_lse(i8, q, s, lse, sl)
            fr.fr_beam_step(beams[0], logits)
            fr.fr_beam_step_lse(beams[1], lse, sl, K)
            a, b = (fr.fr_beam_outputs(x, B, K, D) for x in beams)
            live = a["live"].cpu()
            logp = torch.log_softmax((q.double().cpu() @ wq.double().cpu().T * s.double().cpu()[:, None] * ws.double().cpu())
                                     .view(B, K, V), -1)
            new = torch.zeros_like(scores)
            for r in range(B):
                n = int(live[r])
                assert n == int(b["live"][r])
                par, tok = a["parent"][r, :n].long().cpu(), a["token"][r, :n].long().cpu()
                new[r, :n] = scores[r, par] + logp[r, par, tok]
                assert torch.all((a["score"][r, :n].double().cpu() - new[r, :n]).abs() <= 1e-4)
                assert torch.all((b["score"][r, :n].double().cpu() - new[r, :n]).abs() <= 1e-4)
                gap = (new[r, 1:n] - new[r, :n - 1]).abs().min() if n > 1 else torch.tensor(1.0)
                if gap > 2e-4:  # no near-tie: the same survivors
                    assert torch.equal(a["prefix"][r, :n], b["prefix"][r, :n])
            scores = new
            # the next step's hidden states: the embeddings of the chosen tokens, dead beams (-1) zeros
            nxt = torch.empty(B * K, d, device="cuda")
            fr.fr_embed_lookup(em, table, a["token"].reshape(-1).contiguous(), nxt)
            hidden = nxt.view(B, K, d)
            if t + 1 < D:  # both beams go on from the same survivors
                st = fr.fr_beam_get_state(beams[0], B, K, D)
                assert fr.fr_beam_set_state(beams[1], t + 1, st["live"], st["prefix"], st["score"], st["kv_slot"]) == fr.FR_OK
        assert fr.fr_embed_status(em) == fr.FR_OK
        assert fr.fr_i8_status(i8) == fr.FR_OK and all(fr.fr_beam_status(x) == fr.FR_OK for x in beams)
    finally:
        for x in beams:
            fr.fr_beam_destroy(x)
        fr.fr_trie_destroy(trie)
        fr.fr_embed_destroy(em)
        fr.fr_i8_destroy(i8)


def test_two_handles_on_two_streams():
    """Overlapping runs with a handle each: the same results as one after the other."""
    torch.manual_seed(1)
    rows, V, d = 400, 3000, 128
    sets = []
    for k in range(2):
        h = torch.randn(rows, d, device="cuda").to(BF16)
        wgt = (torch.randn(V, d, device="cuda") * 0.2).to(BF16)
        t = torch.randint(0, V, (rows,), device="cuda", dtype=torch.int32)
        ce = fr.fr_ce_init(V, d, rows)
        loss, lse, gl = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda"), torch.rand(rows, device="cuda")
        dh, dw = torch.empty_like(h), torch.empty_like(wgt)
        sets.append((ce, h, wgt, t, loss, lse, gl, dh, dw))

    def run(ce, h, wgt, t, loss, lse, gl, dh, dw):
        fr.fr_ce_loss(ce, h, wgt, t, loss, lse)
        fr.fr_ce_grad(ce, h, wgt, t, lse, gl, dh, dw)

    want = []
    for s in sets:
        run(*s)
        want.append([x.clone() for x in (s[4], s[7], s[8])])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        for s in sets:
            s[7].zero_(), s[8].zero_()
        torch.cuda.synchronize()
        for st, s in zip(streams, sets):
            with torch.cuda.stream(st):
                run(*s)
        torch.cuda.synchronize()
        for s, wnt in zip(sets, want):
            assert fr.fr_ce_status(s[0]) == fr.FR_OK
            assert all(torch.equal(x, y) for x, y in zip((s[4], s[7], s[8]), wnt))
    for s in sets:
        fr.fr_ce_destroy(s[0])


def _queued():
    """Work on the default stream that is still running when the caller goes on."""
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)  # about 0.2 s


@pytest.mark.parametrize("which", ["embed", "ce", "i8", "lmhead"])
def test_an_error_of_a_run_right_after_init(which):
    """A handle made while the default stream is busy and used on another stream at
    once: what that run records is there to read, and a run without an error
    leaves nothing."""
    rows, V, d = 4, 70, 32
    g = torch.Generator().manual_seed(0)
    bad_tok = torch.tensor([1, V, 2, 3], dtype=torch.int32, device="cuda")
    good_tok = torch.tensor([1, 5, 2, 3], dtype=torch.int32, device="cuda")
    good = torch.randn(rows, d, generator=g).to(BF16).cuda()
    bad = good.clone()
    bad[2, 3] = float("nan")
    table = torch.randn(V, d, generator=g).to(BF16).cuda()
    wq, ws = torch.ones(V, d, dtype=torch.int8, device="cuda"), torch.ones(V, device="cuda")
    xq, good_s = torch.ones(rows, d, dtype=torch.int8, device="cuda"), torch.ones(rows, device="cuda")
    bad_s = good_s.clone()
    bad_s[1] = float("nan")
    out, loss, lse = torch.empty(rows, d, device="cuda"), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    side = torch.cuda.Stream()
    make, run, status, destroy = {
        "embed": (lambda: fr.fr_embed_init(V, d, rows), lambda h, wrong: fr.fr_embed_lookup(h, table, bad_tok if wrong else good_tok, out, stream=side),
                  fr.fr_embed_status, fr.fr_embed_destroy),
        "ce": (lambda: fr.fr_ce_init(V, d, rows), lambda h, wrong: fr.fr_ce_loss(h, good, table, bad_tok if wrong else good_tok, loss, lse, stream=side),
               fr.fr_ce_status, fr.fr_ce_destroy),
        "i8": (lambda: fr.fr_i8_init(wq, ws, rows), lambda h, wrong: fr.fr_i8_lse(h, xq, bad_s if wrong else good_s, lse, None, stream=side),
               fr.fr_i8_status, fr.fr_i8_destroy),
        "lmhead": (lambda: fr.fr_lmhead_init(table, rows, 0, 0), lambda h, wrong: fr.fr_lmhead_run(h, bad if wrong else good, lse, None, stream=side),
                   fr.fr_lmhead_status, fr.fr_lmhead_destroy),
    }[which]
    want = fr.FR_ERR_CODE_RANGE if which in ("embed", "ce") else fr.FR_ERR_NAN_LOGIT
    for wrong in (None, True, False):  # (first with nothing queued: a kernel's first launch loads it, which may wait)
        if wrong is not None:
            _queued()
        h = make()
        try:
            run(h, wrong)
            side.synchronize()
            torch.cuda.synchronize()
            assert status(h) == (want if wrong else fr.FR_OK), wrong
        finally:
            destroy(h)


def test_every_call_refuses_tensors_on_the_cpu():
    rows, V, d = 4, 32, 16
    em, ce = fr.fr_embed_init(V, d, rows), fr.fr_ce_init(V, d, rows)
    wq, ws = torch.ones(V, d, dtype=torch.int8, device="cuda"), torch.ones(V, device="cuda")
    i8 = fr.fr_i8_init(wq, ws, rows, 0, 8)
    table, h = torch.zeros(V, d, dtype=BF16, device="cuda"), torch.zeros(rows, d, dtype=BF16, device="cuda")
    tok, f = torch.zeros(rows, dtype=torch.int32, device="cuda"), torch.zeros(rows, device="cuda")
    xq, out, sl = torch.zeros(rows, d, dtype=torch.int8, device="cuda"), torch.zeros(rows, V, device="cuda"), torch.zeros(rows, 8, device="cuda")
    calls = [
        (fr.fr_embed_lookup, em, (table, tok, h)), (fr.fr_embed_grad, em, (h, tok, table)),
        (fr.fr_ce_loss, ce, (h, table, tok, f, f)), (fr.fr_ce_grad, ce, (h, table, tok, f, f, h, table)),
        (fr.fr_i8_quantize, None, (h, xq, f)), (fr.fr_i8_init, None, (wq, ws)),
        (fr.fr_i8_matmul, i8, (xq, f, out)), (fr.fr_i8_lse, i8, (xq, f, f, sl)),
    ]
    try:
        for call, handle, args in calls:
            for k in range(len(args)):
                moved = [a.cpu() if j == k else a for j, a in enumerate(args)]
                tail = (rows,) if call is fr.fr_i8_init else ()
                with pytest.raises(ValueError, match="CUDA"):
                    call(*(() if handle is None else (handle,)), *moved, *tail)
    finally:
        fr.fr_embed_destroy(em)
        fr.fr_ce_destroy(ce)
        fr.fr_i8_destroy(i8)
