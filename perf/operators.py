"""The vocabulary operators: what each is measured on, and its plain form.

Three operators at the two ends of a generative recommender, around the beam
step: the embedding of the tokens a step chose and its gradient, the softmax
cross entropy of the lm_head projection with its gradients, and the lm_head
product in 8-bit integers.  Sizes are those of the package's own workloads
(V = 151,936, hidden size 2,048, 32 requests x 256 beams, 128 x 50 beams, SID
ranges of 3 x 256 and 5 x 1,024 codes) and ragged ones next to them.

`own` selects the package's kernels; otherwise `run` computes the plain form
in 32 bits and rounds once at the end.
"""
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # the tokens that one serving step chose for 32 x 256 beams, dead beams among them
        dict(name="lookup beams", op="lookup", n=8192, V=151936, d=2048, table="bf16", out="bf16", span=768, dead=0.1),
        # the same for a few beams of one small request, out of a float32 table of odd width
        dict(name="lookup few f32", op="lookup", n=37, V=5151, d=513, table="f32", out="f32", span=0, dead=0.0),
        # a training batch of SID sequences: the tokens fall on few hot rows of a large table
        dict(name="embed grad train", op="embed_grad", n=32768, V=151936, d=2048, grad="bf16", table="bf16", span=768, dead=0.02, add=False),
        # a small tied float32 table: the tokens' gradient is added to what the loss left there
        dict(name="embed grad tied f32", op="embed_grad", n=777, V=5151, d=129, grad="f32", table="f32", span=0, dead=0.1, add=True),
        # a training step's loss and gradients over the whole vocabulary
        dict(name="loss train", op="loss_grad", rows=8192, V=151936, d=2048, ignored=0.05),
        # a fine-tuning step on a few tokens: bound by the weight's bytes
        dict(name="loss few rows", op="loss_grad", rows=96, V=151936, d=2048, ignored=0.0),
        # a loss over the SID range alone (5 x 1,024 codes), ragged, with padded rows
        dict(name="loss sid range", op="loss_grad", rows=6400, V=5120, d=1000, ignored=0.3),
        # an evaluation pass: the loss without gradients
        dict(name="loss eval", op="loss", rows=2048, V=151936, d=2048, ignored=0.05),
        # the first step's root rows, one request: one hidden state by the whole 8-bit lm_head
        dict(name="int8 one token", op="int8", rows=1, N=151936, d=2048, x="bf16", out="bf16"),
        # the logits of a whole serving step
        dict(name="int8 beams", op="int8", rows=8192, N=151936, d=2048, x="bf16", out="bf16"),
        # the serving step's rows as log-sum-exp and SID slice
        dict(name="int8 beams lse", op="int8_lse", rows=8192, N=151936, d=2048, x="bf16", base=131072, span=768),
        # a ragged product with float32 in and out
        dict(name="int8 ragged f32", op="int8", rows=333, N=1003, d=521, x="f32", out="f32"),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["lookup", "embed_grad", "loss_grad", "loss", "int8", "int8_lse"])
    V = _log(rng, 64, 151936)
    if op in ("lookup", "embed_grad"):
        span = rng.choice([0, min(V, _log(rng, 8, 5120))])
        c = dict(op=op, n=_log(rng, 1, 32768), V=V, d=_log(rng, 8, 2048), table=rng.choice(["f32", "bf16"]), span=span, dead=rng.choice([0.0, 0.1, 0.5]))
        if op == "lookup":
            return dict(c, out=rng.choice(["f32", "bf16"]))
        return dict(c, grad=rng.choice(["f32", "bf16"]), add=rng.random() < 0.5)
    rows, d = _log(rng, 1, 8192), _log(rng, 16, 2048)
    if op in ("loss_grad", "loss"):
        return dict(op=op, rows=rows, V=V, d=d, ignored=rng.choice([0.0, 0.1, 0.6]))
    x = rng.choice(["f32", "bf16"])
    if op == "int8":
        out = rng.choice(["f32", "bf16"])  # at most the bytes of a serving step's logits in bf16
        return dict(op=op, rows=rows if out == "bf16" else max(1, rows // 2), N=V, d=d, x=x, out=out)
    span = rng.randint(1, min(V, 5120))
    return dict(op=op, rows=rows, N=V, d=d, x=x, base=rng.randint(0, V - span), span=span)


class _Handle:
    """A library handle that is destroyed with the state that keeps it."""

    def __init__(self, h, destroy):
        self.h, self.destroy = h, destroy

    def __del__(self):
        self.destroy(self.h)


def _padded(rows, cols, dtype, quantum):
    """[rows, cols] whose row pitch is a multiple of `quantum` elements."""
    return torch.empty(rows, -(-cols // quantum) * quantum, dtype=dtype, device="cuda")[:, :cols]


def _normal(gen, rows, cols, dtype, quantum, scale=1.0):
    t = _padded(rows, cols, dtype, quantum)
    t.copy_(torch.randn(rows, cols, device="cuda", generator=gen, dtype=torch.float32 if dtype == torch.float32 else dtype) * scale)
    return t


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, s = case["op"], dict(case=case)
    if op in ("lookup", "embed_grad"):
        n, V, d = case["n"], case["V"], case["d"]
        # a SID batch's tokens lie in the SID range, the heavier codes first; text spreads over the vocabulary
        u = torch.rand(n, device="cuda", generator=gen)
        span = case["span"] or V
        t = ((V - span) + (u * u * span).long().clamp_(max=span - 1)).int()
        s["tokens"] = torch.where(torch.rand(n, device="cuda", generator=gen) < case["dead"], -1, t).int()
        s["scale"] = d ** 0.5
        if op == "lookup":
            s["table"] = _normal(gen, V, d, DTYPES[case["table"]], 1, 0.02)
            s["out"] = torch.empty(n, d, dtype=DTYPES[case["out"]], device="cuda")
        else:
            s["grad"] = _normal(gen, n, d, DTYPES[case["grad"]], 1)
            # what a tied loss left in the table's gradient (read where the tokens' gradient is added)
            s["before"] = _normal(gen, V, d, DTYPES[case["table"]], 1) if case["add"] else None
            s["out"] = torch.empty(V, d, dtype=DTYPES[case["table"]], device="cuda")
    elif op in ("loss", "loss_grad"):
        rows, V, d = case["rows"], case["V"], case["d"]
        s["hidden"] = _normal(gen, rows, d, torch.bfloat16, 8)
        s["weight"] = _normal(gen, V, d, torch.bfloat16, 8, 2.0 * d ** -0.5)
        t = torch.randint(0, V, (rows,), device="cuda", generator=gen, dtype=torch.int32)
        s["targets"] = torch.where(torch.rand(rows, device="cuda", generator=gen) < case["ignored"], -1, t).int()
        s["loss"] = torch.empty(rows, device="cuda")
        s["lse"] = torch.empty(rows, device="cuda")
        if op == "loss_grad":
            # the mean over the rows that count, times a loss scale
            s["grad_loss"] = torch.full((rows,), 64.0, device="cuda") / (s["targets"] >= 0).sum().clamp(min=1)
            s["grad_hidden"] = torch.empty(rows, d, dtype=torch.bfloat16, device="cuda")
            s["grad_weight"] = torch.empty(V, d, dtype=torch.bfloat16, device="cuda")
    else:
        rows, N, d = case["rows"], case["N"], case["d"]
        s["x"] = _normal(gen, rows, d, DTYPES[case["x"]], 1)
        # the weight as a program keeps it: symmetric 8 bits with a scale for each output channel
        w = torch.randn(N, d, device="cuda", generator=gen) * (2.0 * d ** -0.5)
        s["ws"] = _step(w)
        s["wq"] = _padded(N, d, torch.int8, 16)
        s["wq"].copy_(torch.round(w / s["ws"][:, None]).to(torch.int8))
        s["xq"], s["xs"] = _padded(rows, d, torch.int8, 16), torch.empty(rows, device="cuda")
        if op == "int8":
            s["out"] = torch.empty(rows, N, dtype=DTYPES[case["out"]], device="cuda")
        else:
            s["lse"], s["slice"] = torch.empty(rows, device="cuda"), torch.empty(rows, case["span"], device="cuda")
    if own:  # the handle that a program keeps
        from trie_constrained_beam_fr_b200 import fr

        s["fr"] = fr
        if op in ("lookup", "embed_grad"):
            s["handle"] = _Handle(fr.fr_embed_init(case["V"], case["d"], case["n"]), fr.fr_embed_destroy)
        elif op in ("loss", "loss_grad"):
            s["handle"] = _Handle(fr.fr_ce_init(case["V"], case["d"], case["rows"]), fr.fr_ce_destroy)
        else:
            s["handle"] = _Handle(fr.fr_i8_init(s["wq"], s["ws"], case["rows"], case.get("base", 0), case.get("span", 0)), fr.fr_i8_destroy)
    return s


def _run_own(s):
    fr, h, op = s["fr"], s["handle"].h, s["case"]["op"]
    if op == "lookup":
        fr.fr_embed_lookup(h, s["table"], s["tokens"], s["out"], s["scale"])
        return s["out"]
    if op == "embed_grad":
        if s["before"] is not None:
            s["out"].copy_(s["before"])
        fr.fr_embed_grad(h, s["grad"], s["tokens"], s["out"], s["scale"], s["before"] is not None)
        return s["out"]
    if op in ("loss", "loss_grad"):
        fr.fr_ce_loss(h, s["hidden"], s["weight"], s["targets"], s["loss"], s["lse"])
        if op == "loss":
            return {"loss": s["loss"], "lse": s["lse"]}
        fr.fr_ce_grad(h, s["hidden"], s["weight"], s["targets"], s["lse"], s["grad_loss"], s["grad_hidden"], s["grad_weight"])
        return {"loss": s["loss"], "lse": s["lse"], "grad_hidden": s["grad_hidden"], "grad_weight": s["grad_weight"]}
    fr.fr_i8_quantize(s["x"], s["xq"], s["xs"])
    if op == "int8":
        fr.fr_i8_matmul(h, s["xq"], s["xs"], s["out"])
        return s["out"]
    fr.fr_i8_lse(h, s["xq"], s["xs"], s["lse"], s["slice"])
    return {"lse": s["lse"], "slice": s["slice"]}


def _step(x):
    """Each row's quantisation step: an IEEE quotient (by a tensor: a division by a number multiplies by its reciprocal)."""
    m = x.abs().amax(1)
    return m / torch.full_like(m, 127.0)


def _row_lse(x):
    m = x.amax(1)
    return m + (x - m[:, None]).exp_().sum(1).log()


def run(s):
    if own:
        return _run_own(s)
    c = s["case"]
    op = c["op"]
    if op in ("lookup", "embed_grad"):
        t = s["tokens"].long()
        live = t >= 0
        if op == "lookup":
            x = s["table"][t.clamp(min=0)].float() * s["scale"]
            return torch.where(live[:, None], x, 0.0).to(s["out"].dtype)
        g = torch.where(live[:, None], s["grad"].float(), 0.0)
        total = torch.zeros(c["V"], c["d"], device="cuda").index_add_(0, t.clamp(min=0), g) * s["scale"]
        if s["before"] is not None:
            total += s["before"].float()
        return total.to(s["out"].dtype)
    if op in ("loss", "loss_grad"):
        h, w, t = s["hidden"].float(), s["weight"].float(), s["targets"].long()
        live, at = t >= 0, t.clamp(min=0)
        x = h @ w.T
        lse = _row_lse(x)
        loss = torch.where(live, lse - x.gather(1, at[:, None])[:, 0], 0.0)
        if op == "loss_grad":
            x.sub_(lse[:, None]).exp_()
        lse = torch.where(live, lse, 0.0)  # rows that do not count
        if op == "loss":
            return {"loss": loss, "lse": lse}
        x.scatter_add_(1, at[:, None], torch.full((len(t), 1), -1.0, device="cuda"))
        x.mul_(torch.where(live, s["grad_loss"], 0.0)[:, None])
        return {"loss": loss, "lse": lse, "grad_hidden": (x @ w).bfloat16(), "grad_weight": (x.T @ h).bfloat16()}
    x = s["x"].float()
    xs = _step(x)
    q = torch.round(x / torch.where(xs > 0, xs, 1.0)[:, None])
    y = q @ s["wq"].float().T
    y *= xs[:, None]
    y *= s["ws"]
    if op == "int8":
        return y.to(s["out"].dtype)
    return {"lse": _row_lse(y), "slice": y[:, c["base"]:c["base"] + c["span"]].clone()}


def work(case):
    op, size = case["op"], {"f32": 4, "bf16": 2}
    if op in ("lookup", "embed_grad"):
        n, V, d = case["n"], case["V"], case["d"]
        live = n * (1 - case["dead"])
        if op == "lookup":
            # rows that several tokens share are read once
            return {"bytes": min(live, case["span"] or V) * d * size[case["table"]] + n * (4 + d * size[case["out"]]), "flops": 0}
        table = V * d * size[case["table"]]
        return {"bytes": n * 4 + live * d * size[case["grad"]] + table * (2 if case["add"] else 1), "flops": live * d}
    if op in ("loss", "loss_grad"):
        rows, V, d = case["rows"] * (1 - case["ignored"]), case["V"], case["d"]  # the rows that count
        inputs, product = 2 * d * (rows + V) + 4 * rows, 2 * rows * V * d
        if op == "loss":
            return {"bytes": inputs + 8 * rows, "flops": product}
        return {"bytes": 2 * inputs + 16 * rows, "flops": 3 * product}
    rows, N, d = case["rows"], case["N"], case["d"]
    inputs = N * (d + 4) + rows * d * size[case["x"]]
    outputs = rows * N * size[case["out"]] if op == "int8" else rows * 4 * (1 + case["span"])
    return {"bytes": inputs + outputs, "flops": 2 * rows * N * d}


def exact(case, seed):
    """The definitions in 64 bits."""
    s, f64 = prepare(case, seed), torch.float64
    op = case["op"]
    if op == "lookup":
        table = torch.cat([s["table"].to(f64) * s["scale"], torch.zeros(1, case["d"], dtype=f64, device="cuda")])
        return table[s["tokens"].long()]  # token -1 is the last row: zeros
    if op == "embed_grad":
        # sorted by token: differences of a running sum would cancel, so the rows of each run are added in turns
        out = torch.zeros(case["V"] + 1, case["d"], dtype=f64, device="cuda")
        order = torch.argsort(s["tokens"], stable=True)
        tok = s["tokens"][order].long()
        start = torch.searchsorted(tok, tok)
        turn = torch.arange(len(tok), device="cuda") - start
        for k in torch.unique(turn).tolist():
            at = turn == k  # the k-th row of every token: no token twice
            out[tok[at]] += s["grad"][order[at]].to(f64)
        out = out[:-1] * s["scale"]
        return out if s["before"] is None else out + s["before"].to(f64)
    if op in ("loss", "loss_grad"):
        h, w, keep = s["hidden"].to(f64), s["weight"].to(f64), s["targets"] >= 0
        logp = torch.mm(h, w.t())
        lse = torch.logsumexp(logp, dim=1)
        logp -= lse[:, None]
        lse *= keep
        rows = torch.nonzero(keep)[:, 0]
        cols = s["targets"][rows].long()
        loss = torch.zeros(len(h), dtype=f64, device="cuda")
        loss[rows] = -logp[rows, cols]
        if op == "loss":
            return {"loss": loss, "lse": lse}
        g = torch.exp(logp)
        del logp
        g[rows, cols] -= 1
        g *= (s["grad_loss"].to(f64) * keep)[:, None]
        return {"loss": loss, "lse": lse, "grad_hidden": torch.mm(g, w), "grad_weight": torch.mm(g.t(), h)}
    # the quantised values are a definition in 32 bits: x / (amax / 127), each rounded to nearest even
    x = s["x"].float()
    step = (x.abs().max(dim=1, keepdim=True).values.to(f64) / 127).float()
    q = torch.where(step == 0, torch.zeros_like(x), torch.round(x / step))
    y = torch.mm(q.to(f64), s["wq"].to(f64).t()) * step.to(f64) * s["ws"].to(f64)[None, :]
    if op == "int8":
        return y
    return {"lse": torch.logsumexp(y, dim=1), "slice": y.narrow(1, case["base"], case["span"]).clone()}
