"""Cases of the operators between a model's logits and its training-state step.

Two operators over rows of logits (one row per token position, `vocab` columns):

* token log probabilities: the log probability of a given token, the entropy,
  the log of the normaliser and the top alternatives of every row, and the
  gradient of all of them with respect to the logits;
* distillation from a teacher's top log probabilities: the divergence of every
  row from k listed (token, log probability) pairs, and its gradient, either in
  the same call or from the saved normalisers (maximum and sum of each row).

`own` selects the side: elementary torch operations in 32 bits, or the
library's calls.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
IDTYPES = {"i32": torch.int32, "i64": torch.int64}


def listed():
    return [
        # serving, one sequence: the sampled token's log probability and five alternatives (GPT-2 vocabulary)
        dict(name="logprobs-1x50257-fp16-top5", op="logprobs", rows=1, vocab=50257, pad=0, dtype="fp16", ids="i64", k=5,
             scale=1.0),
        # serving, eight sequences decoding together, twenty alternatives (Llama-3 vocabulary), temperature 0.7
        dict(name="logprobs-8x128256-bf16-top20", op="logprobs", rows=8, vocab=128256, pad=0, dtype="bf16", ids="i64",
             k=20, scale=1.0 / 0.7),
        # evaluation of a small model that keeps fp32 logits, an odd number of positions
        dict(name="logprobs-1021x50257-fp32-top20", op="logprobs", rows=1021, vocab=50257, pad=0, dtype="fp32",
             ids="i64", k=20, scale=1.0),
        # scoring a batch of rollouts: log probabilities and entropies only
        dict(name="logprobs-4096x128256-bf16-top0", op="logprobs", rows=4096, vocab=128256, pad=0, dtype="bf16",
             ids="i64", k=0, scale=1.0),
        # a teacher's pass that stores its top 64 log probabilities for distillation
        dict(name="logprobs-2048x128256-bf16-top64", op="logprobs", rows=2048, vocab=128256, pad=0, dtype="bf16",
             ids="i32", k=64, scale=1.0),
        # policy-gradient update with an entropy bonus and a penalty on the normaliser
        dict(name="logprobs_grad-2048x128256-bf16", op="logprobs_grad", rows=2048, vocab=128256, pad=0, dtype="bf16",
             ids="i64", k=0, scale=1.0),
        # gradient of the token and of eight alternatives, fp32 logits, odd rows
        dict(name="logprobs_grad-509x50257-fp32-top8", op="logprobs_grad", rows=509, vocab=50257, pad=0, dtype="fp32",
             ids="i64", k=8, scale=1.0),
        # held-out distillation loss of a small student, fp16 logits, no gradient
        dict(name="distill_loss-1024x50257-fp16-top16", op="distill_loss", rows=1024, vocab=50257, pad=0, dtype="fp16",
             ids="i32", k=16, scale=1.0, tail="renorm"),
        # distillation step of a Llama-3-vocabulary student: loss and gradient in one call, rest of the mass in a bucket
        dict(name="distill-4096x128256-bf16-top64", op="distill", rows=4096, vocab=128256, pad=0, dtype="bf16",
             ids="i32", k=64, scale=1.0, tail="bucket"),
        # the same for a GPT-2-vocabulary student, its head padded to 50304 columns; every eighth position is padding
        dict(name="distill-999x50257-bf16-top32", op="distill", rows=999, vocab=50257, pad=47, dtype="bf16",
             ids="i64", k=32, scale=0.5, tail="renorm", skip=8),
        # a micro-batch with fp32 logits and the longest list
        dict(name="distill-64x128256-fp32-top128", op="distill", rows=64, vocab=128256, pad=0, dtype="fp32", ids="i32",
             k=128, scale=1.0, tail="bucket"),
        # backward of a separate forward: the gradient from the saved normalisers
        dict(name="distill_grad-2048x128256-bf16-top64", op="distill_grad", rows=2048, vocab=128256, pad=0,
             dtype="bf16", ids="i32", k=64, scale=1.0, tail="bucket"),
    ]


_MOST = 4096 * 128256 * 2  # bytes of the largest listed case's logits


def draw(rng):
    def log_between(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["logprobs", "logprobs", "logprobs_grad", "distill_loss", "distill", "distill", "distill_grad"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    vocab = rng.choice([50257, 128256, log_between(1000, 200000), log_between(1000, 200000)])
    most = max(1, min(8192, _MOST // (vocab * (4 if dtype == "fp32" else 2))))
    case = dict(op=op, rows=log_between(1, most), vocab=vocab,
                pad=rng.choice([0, 0, -vocab % 64, rng.randrange(1, 100)]), dtype=dtype,
                ids=rng.choice(["i32", "i64"]), scale=rng.choice([1.0, 1.0, 0.5, 1.0 / 0.7]))
    if op.startswith("logprobs"):
        case["k"] = rng.choice([0, 1, log_between(1, 128), log_between(1, 128)])
    else:
        case["k"] = log_between(1, 128)
        case["tail"] = rng.choice(["drop", "renorm", "bucket"])
        case["skip"] = rng.choice([0, 0, 8])
    return case


# ------------------------------------------------------------------ inputs

def _logits(case, gen, dev):
    """Rows of logits: a broad bulk and some favoured tokens a few units above it, as a language model's head gives."""
    rows, vocab, pad = case["rows"], case["vocab"], case["pad"]
    x = torch.empty((rows, vocab + pad), dtype=DTYPES[case["dtype"]], device=dev)
    step = max(1, (1 << 27) // vocab)
    for r in range(0, rows, step):
        n = min(step, rows - r)
        z = torch.randn((n, vocab), generator=gen, device=dev).mul_(2.0)
        fav = torch.randint(0, vocab, (n, 48), generator=gen, device=dev)
        z.scatter_add_(1, fav, torch.rand((n, 48), generator=gen, device=dev) * 11.0)
        x[r:r + n, :vocab] = z
    if pad:
        x[:, vocab:] = 0
    return x[:, :vocab]


def _top(x, k):
    """(values, ids) of the k largest of each row in descending order, equal values by ascending id."""
    b = (x.float() + 0.0).view(torch.int32).to(torch.int64)
    key = torch.where(b < 0, b ^ 0x7FFFFFFF, b)
    key = key * (1 << 32) + ((1 << 32) - 1 - torch.arange(x.shape[1], device=x.device))
    key = torch.topk(key, k, dim=1, sorted=True).values
    ids = (1 << 32) - 1 - (key & 0xFFFFFFFF)
    return x.float().gather(1, ids), ids


def _teacher(case, x, gen):
    """A teacher that differs from the student by noise: its top k ids and log probabilities, by chunks of rows."""
    ids, lps = [], []
    step = max(1, (1 << 26) // case["vocab"])
    for r in range(0, case["rows"], step):
        z = x[r:r + step].float() * case["scale"]
        z += torch.randn(z.shape, generator=gen, device=z.device).mul_(0.5)
        v, i = torch.topk(z, min(case["k"], case["vocab"]), dim=1)
        ids.append(i)
        lps.append(v - torch.logsumexp(z, dim=1, keepdim=True))
    return torch.cat(ids).to(IDTYPES[case["ids"]]), torch.cat(lps)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    rows, vocab, k, op = case["rows"], case["vocab"], case["k"], case["op"]
    x = _logits(case, gen, dev)
    s = {"case": case, "x": x, "scale": case["scale"]}
    f32 = dict(dtype=torch.float32, device=dev)
    idt = IDTYPES[case["ids"]]
    if op.startswith("logprobs"):
        # most given tokens are likely ones; every seventh row is any token
        likely = x[:, :min(vocab, 4096)].argmax(dim=1)
        anyone = torch.randint(0, vocab, (rows,), generator=gen, device=dev)
        r = torch.arange(rows, device=dev)
        s["tokens"] = torch.where(r % 7 == 3, anyone, likely).to(idt)
        if op == "logprobs":
            s["out"] = {n: torch.empty(rows, **f32) for n in ("logprob", "entropy", "lse")}
            if k:
                s["out"]["top_logprob"] = torch.empty((rows, k), **f32)
                s["out"]["top_id"] = torch.empty((rows, k), dtype=idt, device=dev)
        else:
            # what a forward saved (the normaliser as the pair of maximum and sum, the entropy, the alternatives), and
            # the upstream gradients: advantages, the bonus, the penalty
            norm = torch.empty((rows, 2), **f32)
            ent = torch.empty(rows, **f32)
            ids = torch.empty((rows, k), dtype=idt, device=dev)
            step = max(1, (1 << 26) // vocab)
            for i in range(0, rows, step):
                z = x[i:i + step].double() * case["scale"]
                m = z.max(dim=1).values
                l = torch.logsumexp(z, dim=1)
                p = torch.exp(z - l[:, None])
                norm[i:i + step, 0] = x[i:i + step].max(dim=1).values
                norm[i:i + step, 1] = torch.exp(l - m)
                ent[i:i + step] = l - (p * z).sum(dim=1)
                if k:
                    ids[i:i + step] = _top(x[i:i + step], k)[1].to(idt)
            s["norm"], s["entropy"], s["top_id"] = norm, ent, ids if k else None
            s["d_logprob"] = torch.randn(rows, generator=gen, **f32) / rows
            s["d_entropy"] = torch.full((rows,), -0.01 / rows, **f32)
            s["d_lse"] = (norm[:, 0] * case["scale"] + torch.log(norm[:, 1])) * (2e-4 / rows)
            s["d_top"] = torch.randn((rows, k), generator=gen, **f32) / rows if k else None
            s["d_logits"] = torch.empty((rows, vocab + case["pad"]), dtype=x.dtype, device=dev)[:, :vocab]
        return s
    s["ids"], s["teacher"] = _teacher(case, x, gen)
    s["tail"] = case["tail"]
    w = torch.full((rows,), 1.0 / rows, **f32)
    if case.get("skip"):
        w[case["skip"] - 1::case["skip"]] = 0.0  # padding positions
    s["weight"] = w
    s["loss"] = torch.empty(rows, **f32)
    s["norm"] = torch.empty((rows, 2), **f32)
    s["tail_logprob"] = torch.empty(rows, **f32)
    if op != "distill_loss":
        s["d_logits"] = torch.empty((rows, vocab + case["pad"]), dtype=x.dtype, device=dev)[:, :vocab]
    if op == "distill_grad":
        s["d_loss"] = torch.rand(rows, generator=gen, **f32) + 0.5
        step = max(1, (1 << 26) // vocab)
        for i in range(0, rows, step):
            z = x[i:i + step].double() * case["scale"]
            l = torch.logsumexp(z, dim=1)
            s["norm"][i:i + step, 0] = x[i:i + step].max(dim=1).values
            s["norm"][i:i + step, 1] = torch.exp(l - z.max(dim=1).values)
            z.scatter_(1, s["ids"][i:i + step].long(), -math.inf)
            s["tail_logprob"][i:i + step] = torch.logsumexp(z, dim=1) - l
    return s


# ------------------------------------------------------------------ the plain form

def _plain_logprobs(s):
    x, c, k = s["x"], s["scale"], s["case"]["k"]
    z = x.float() * c
    m = z.max(dim=1, keepdim=True).values
    d = z - m
    e = torch.exp(d)
    t = e.sum(dim=1)
    log_t = torch.log(t)
    out = {"logprob": d.gather(1, s["tokens"].long()[:, None])[:, 0] - log_t,
           "entropy": log_t - (e * d).sum(dim=1) / t, "lse": m[:, 0] + log_t}
    if k:
        v, ids = _top(x, k)
        out["top_logprob"] = (v * c - m) - log_t[:, None]
        out["top_id"] = ids.to(s["tokens"].dtype)
    return out


def _plain_logprobs_grad(s):
    x, c, k = s["x"], s["scale"], s["case"]["k"]
    z = x.float() * c
    d = z - z.max(dim=1, keepdim=True).values
    e = torch.exp(d)
    t = e.sum(dim=1, keepdim=True)
    p = e / t
    logp = d - torch.log(t)
    total = s["d_logprob"] - s["d_lse"]
    if k:
        total = total + s["d_top"].sum(dim=1)
    g = -p * total[:, None] - (s["d_entropy"][:, None] * p) * (logp + s["entropy"][:, None])
    g.scatter_add_(1, s["tokens"].long()[:, None], s["d_logprob"][:, None])
    if k:
        g.scatter_add_(1, s["top_id"].long(), s["d_top"])
    return {"d_logits": (g * c).to(x.dtype)}


def _plain_distill(s, want_grad, d_loss=None):
    x, c, mode, w = s["x"], s["scale"], s["tail"], s["weight"]
    ids = s["ids"].long()
    logq = s["teacher"].float()
    if mode == "renorm":
        logq = logq - torch.log(torch.exp(logq).sum(dim=1, keepdim=True))
    q = torch.exp(logq)
    z = x.float() * c
    m = z.max(dim=1, keepdim=True).values
    d = z - m
    e = torch.exp(d)
    t = e.sum(dim=1, keepdim=True)
    logp = d.gather(1, ids) - torch.log(t)
    loss = (q * (logq - logp)).sum(dim=1)
    qsum = q.sum(dim=1)
    rest = e.scatter(1, ids, 0.0).sum(dim=1, keepdim=True)
    tail_logp = (torch.log(rest) - torch.log(t))[:, 0]
    if mode == "bucket":
        qt = (1.0 - qsum).clamp_min(0.0)
        loss = loss + torch.where(qt > 0, qt * (torch.log(qt) - tail_logp), 0.0)
    live = w != 0
    if not want_grad:
        norm = torch.cat([x.max(dim=1, keepdim=True).values.float(), t], dim=1)
        out = {"loss": torch.where(live, loss * w, 0.0), "norm": torch.where(live[:, None], norm, 0.0)}
        if mode == "bucket":
            out["tail_logprob"] = torch.where(live, tail_logp, 0.0)
        return out
    p = e / t
    if mode == "bucket":
        g = p - (qt[:, None] / rest) * e
        b = qsum + qt
    else:
        g = p * qsum[:, None]
        b = qsum
    g.scatter_(1, ids, p.gather(1, ids) * b[:, None] - q)
    g = g * (w * c)[:, None]
    if d_loss is not None:
        g = g * d_loss[:, None]
    g = torch.where(live[:, None], g, 0.0).to(x.dtype)
    return {"d_logits": g} if d_loss is not None else {"loss": torch.where(live, loss * w, 0.0), "d_logits": g}


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if not own:
        if op == "logprobs":
            return _plain_logprobs(s)
        if op == "logprobs_grad":
            return _plain_logprobs_grad(s)
        if op == "distill_grad":
            return _plain_distill(s, True, s["d_loss"])
        return _plain_distill(s, op == "distill")
    import fsdp_sharded_mixed_ss_gb300 as ss

    if op == "logprobs":
        ss.ss_token_logprobs(s["x"], s["tokens"], scale=s["scale"], **s["out"])
        return s["out"]
    if op == "logprobs_grad":
        ss.ss_token_logprobs_grad(s["x"], s["norm"], s["d_logits"], tokens=s["tokens"], d_logprob=s["d_logprob"],
                                  entropy=s["entropy"], d_entropy=s["d_entropy"], d_lse=s["d_lse"],
                                  top_id=s["top_id"], d_top_logprob=s["d_top"], scale=s["scale"])
        return {"d_logits": s["d_logits"]}
    tail = {"drop": ss.SS_TAIL_DROP, "renorm": ss.SS_TAIL_RENORM, "bucket": ss.SS_TAIL_BUCKET}[s["tail"]]
    if op == "distill_grad":
        ss.ss_distill_topk_grad(s["x"], s["ids"], s["teacher"], s["norm"], s["d_logits"],
                                tail_logprob=s["tail_logprob"], d_loss=s["d_loss"], row_weight=s["weight"], tail=tail,
                                scale=s["scale"])
        return {"d_logits": s["d_logits"]}
    if op == "distill":
        ss.ss_distill_topk(s["x"], s["ids"], s["teacher"], s["loss"], d_logits=s["d_logits"], row_weight=s["weight"],
                           tail=tail, scale=s["scale"])
        return {"loss": s["loss"], "d_logits": s["d_logits"]}
    out = {"loss": s["loss"], "norm": s["norm"]}
    if s["tail"] == "bucket":
        out["tail_logprob"] = s["tail_logprob"]
    ss.ss_distill_topk(s["x"], s["ids"], s["teacher"], row_weight=s["weight"], tail=tail, scale=s["scale"], **out)
    return out


def work(case):
    """Each input once and each output once. A skipped row of a distillation is not read; its gradient is written."""
    rows, vocab, k, op = case["rows"], case["vocab"], case["k"], case["op"]
    es = 4 if case["dtype"] == "fp32" else 2
    ib = 4 if case["ids"] == "i32" else 8
    live = rows - rows // case["skip"] if case.get("skip") else rows
    n, read = rows * vocab, live * vocab
    if op == "logprobs":
        return {"bytes": n * es + rows * (ib + 12 + k * (4 + ib)), "flops": 7 * n}
    if op == "logprobs_grad":
        return {"bytes": 2 * n * es + rows * (ib + 24 + k * (4 + ib)), "flops": 6 * n}
    lists = live * k * (4 + ib) + rows * 4
    if op == "distill_loss":
        return {"bytes": read * es + lists + rows * (16 if case["tail"] == "bucket" else 12), "flops": 4 * read}
    if op == "distill":
        return {"bytes": (read + n) * es + lists + rows * 4, "flops": 8 * read}
    return {"bytes": (read + n) * es + lists + rows * 16, "flops": 4 * read}


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    """From the definitions, on float64 rows: softmax by torch's own normalisers of single rows' worth of work, the
    divergence as a sum over every listed pair, and the gradients as products with the softmax's Jacobian."""
    s = prepare(case, seed)
    x, c, k, op = s["x"], float(s["scale"]), case["k"], case["op"]
    rows, vocab = case["rows"], case["vocab"]
    step = max(1, (1 << 25) // vocab)
    parts = []
    for r in range(0, rows, step):
        sl = slice(r, min(rows, r + step))
        logp = torch.log_softmax(x[sl].double() * c, dim=1)
        p = logp.exp()
        if op.startswith("logprobs"):
            tok = s["tokens"][sl].long()[:, None]
            entropy = -(p * logp).sum(dim=1)
            if op == "logprobs":
                o = {"logprob": logp.gather(1, tok)[:, 0], "entropy": entropy,
                     "lse": torch.logsumexp(x[sl].double() * c, dim=1)}
                if k:
                    # descending, equal values by ascending id: a stable sort of the values themselves
                    order = torch.sort(x[sl].double(), dim=1, descending=True, stable=True).indices[:, :k]
                    o["top_logprob"] = logp.gather(1, order)
                    o["top_id"] = order.to(s["tokens"].dtype)
                parts.append(o)
                continue
            # upstream gradient of logp (token, alternatives, entropy's own log), then through log_softmax
            v = torch.zeros_like(p)
            v.scatter_add_(1, tok, s["d_logprob"][sl].double()[:, None])
            if k:
                v.scatter_add_(1, s["top_id"][sl].long(), s["d_top"][sl].double())
            v -= s["d_entropy"][sl].double()[:, None] * p * (logp + 1.0)
            g = v - p * v.sum(dim=1, keepdim=True) + p * s["d_lse"][sl].double()[:, None]
            parts.append({"d_logits": g * c})
            continue
        ids = s["ids"][sl].long()
        w = s["weight"][sl].double()
        lq = s["teacher"][sl].double()
        if case["tail"] == "renorm":
            lq = torch.log_softmax(lq, dim=1)
        q = lq.exp()
        lp = logp.gather(1, ids)
        loss = (q * lq - q * lp).sum(dim=1)
        # v: gradient of the loss with respect to the probabilities' logs
        v = torch.zeros_like(p).scatter_add_(1, ids, -q)
        if case["tail"] == "bucket":
            qt = (1.0 - q.sum(dim=1)).clamp_min(0.0)
            outside = torch.ones_like(p).scatter_(1, ids, 0.0)
            pt = (p * outside).sum(dim=1)
            loss = loss + torch.where(qt > 0, qt * (qt.clamp_min(1e-300).log() - pt.log()), 0.0)
            v -= (qt / pt)[:, None] * p * outside
        o = {"loss": loss * w}
        if op == "distill_loss":
            live = w != 0
            big = x[sl].double().max(dim=1).values
            o["norm"] = torch.where(live[:, None], torch.stack(
                [big, ((x[sl].double() - big[:, None]) * c).exp().sum(dim=1)], dim=1), 0.0)
            if case["tail"] == "bucket":
                o["tail_logprob"] = torch.where(live, pt.log(), 0.0)
        else:
            g = (v - p * v.sum(dim=1, keepdim=True)) * (c * w)[:, None]
            if op == "distill_grad":
                g = g * s["d_loss"][sl].double()[:, None]
                o = {}
            o["d_logits"] = g
        parts.append(o)
    return {n: torch.cat([o[n] for o in parts]) for n in parts[0]}
