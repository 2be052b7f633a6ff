"""Cases of the operators at a model's two vocabulary ends: its losses on sampled tokens, and its embedding.

* policy: the clipped policy loss of every row of logits (one row per token position, `vocab` columns), with a KL term
  against a reference model and an entropy bonus, and the gradient with respect to the logits in the same call;
* policy_loss: the same without the gradient, with what a separate backward pass takes;
* preference: the loss of pairs of sequences (chosen, rejected) from their tokens' log probabilities, and its gradient
  with respect to them;
* embedding: rows of a table by token, scaled;
* embedding_grad: the table's gradient, the sum of each token's occurrences, on top of what is there already.

`own` selects the side: elementary torch operations in 32 bits (64 for ratios next to a border of the clipping and for
long sums), or the library's calls.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
IDTYPES = {"i32": torch.int32, "i64": torch.int64}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4, "i32": 4, "i64": 8}


def listed():
    return [
        # a micro-batch's first update on fresh samples of a GPT-2-vocabulary policy: no old policy yet, no reference
        dict(name="policy-24x50257-fp16", op="policy", rows=24, vocab=50257, pad=0, dtype="fp16", ids="i64", old=False,
             kl="none", kl_coef=0.0, entropy=0.0, dual=0.0, skip=0, scale=1.0),
        # a step on 4096 sampled tokens of a Llama-3-vocabulary policy, KL term against the reference model
        dict(name="policy-4096x128256-bf16-kl", op="policy", rows=4096, vocab=128256, pad=0, dtype="bf16", ids="i64",
             old=True, kl="k3", kl_coef=0.04, entropy=0.0, dual=0.0, skip=0, scale=1.0),
        # fp32 logits of a padded head, an odd number of positions of which a third are prompts, entropy bonus, bounded
        # loss of negative advantages, temperature 0.8
        dict(name="policy-1021x50257-fp32-entropy", op="policy", rows=1021, vocab=50257, pad=47, dtype="fp32",
             ids="i32", old=True, kl="k2", kl_coef=0.1, entropy=0.01, dual=3.0, skip=3, scale=1.25),
        # the forward pass alone, with what a backward pass of its own takes
        dict(name="policy_loss-2048x128256-bf16", op="policy_loss", rows=2048, vocab=128256, pad=0, dtype="bf16",
             ids="i64", old=True, kl="k1", kl_coef=0.05, entropy=0.01, dual=0.0, skip=0, scale=1.0),
        # four pairs of answers of a few hundred tokens: a micro-batch
        dict(name="preference-4x2911", op="preference", pairs=4, tokens=2911, behind=0, ids="i64", kind="sigmoid",
             smooth=0.0, average=False, ref=True, halves=False),
        # a batch of long answers, chosen ones first, without a reference model: mean log probabilities and a margin
        dict(name="preference-256x401023-average", op="preference", pairs=256, tokens=401023, behind=129, ids="i32",
             kind="hinge", smooth=0.0, average=True, ref=False, halves=True),
        # a whole epoch's log probabilities at once
        dict(name="preference-2048x6291456", op="preference", pairs=2048, tokens=6291456, behind=0, ids="i64",
             kind="sigmoid", smooth=0.1, average=False, ref=True, halves=False),
        # the tokens of 96 sequences decoding together, a 4096-wide model
        dict(name="embedding-96x4096-bf16", op="embedding", n=96, vocab=128256, dim=4096, dtype="bf16", out="bf16",
             ids="i64", scale=1.0, holes=0),
        # a prompt batch, rows scaled by the root of the width, some positions padding
        dict(name="embedding-16381x4096-bf16", op="embedding", n=16381, vocab=128256, dim=4096, dtype="bf16",
             out="bf16", ids="i32", scale=64.0, holes=9),
        # a GPT-2 micro-batch, fp16, an odd number of tokens
        dict(name="embedding_grad-1013x768-fp16", op="embedding_grad", n=1013, vocab=50257, dim=768, dtype="fp16",
             out="fp16", ids="i64", scale=1.0, holes=0, base="none"),
        # a tied table: the tokens' part on top of the head's fp32 gradient, rounded once into the unit's 16-bit gradient
        dict(name="embedding_grad-16384x768-bf16-tied", op="embedding_grad", n=16384, vocab=50257, dim=768,
             dtype="bf16", out="bf16", ids="i32", scale=1.0, holes=0, base="fp32"),
        # a large batch of a Llama-3-vocabulary model
        dict(name="embedding_grad-65536x4096-bf16", op="embedding_grad", n=65536, vocab=128256, dim=4096, dtype="bf16",
             out="bf16", ids="i64", scale=1.0, holes=9, base="none"),
    ]


_MOST = 4096 * 128256 * 2  # bytes of the largest listed case's logits


def draw(rng):
    def log_between(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["policy", "policy", "policy_loss", "preference", "embedding", "embedding_grad", "embedding_grad"])
    ids = rng.choice(["i32", "i64"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    vocab = rng.choice([50257, 128256, log_between(1000, 200000), log_between(1000, 200000)])
    if op.startswith("policy"):
        most = max(1, min(8192, _MOST // (vocab * BYTES[dtype])))
        kl = rng.choice(["none", "k1", "k2", "k3"])
        return dict(op=op, rows=log_between(1, most), vocab=vocab,
                    pad=rng.choice([0, 0, -vocab % 64, rng.randrange(1, 100)]), dtype=dtype, ids=ids,
                    old=rng.random() < 0.75, kl=kl, kl_coef=0.0 if kl == "none" else rng.choice([0.01, 0.04, 0.1]),
                    entropy=rng.choice([0.0, 0.0, 0.001, 0.01]), dual=rng.choice([0.0, 0.0, 3.0]),
                    skip=rng.choice([0, 0, 3, 8]), scale=rng.choice([1.0, 1.0, 0.5, 1.25]))
    if op == "preference":
        pairs = log_between(1, 2048)
        return dict(op=op, pairs=pairs, tokens=log_between(2 * pairs, min(6291456, 32768 * pairs)),
                    behind=rng.choice([0, 0, rng.randrange(1, 1000)]), ids=ids,
                    kind=rng.choice(["sigmoid", "sigmoid", "hinge", "square"]), smooth=rng.choice([0.0, 0.1]),
                    average=rng.random() < 0.5, ref=rng.random() < 0.7, halves=rng.random() < 0.5)
    dim = rng.choice([128, 256, 512, 768, 4096, 8192, log_between(64, 8192), log_between(64, 8192)])
    vocab = min(vocab, 128256 * 4096 * 2 // (dim * BYTES[dtype]))
    most = min(65536, 65536 * 4096 * 2 // (dim * BYTES[dtype]))
    case = dict(op=op, n=log_between(1, most), vocab=vocab, dim=dim, dtype=dtype, out=rng.choice([dtype, "bf16"]),
                ids=ids, scale=rng.choice([1.0, 1.0, 0.125, 64.0]), holes=rng.choice([0, 0, 9]))
    if op == "embedding_grad":
        case["base"] = rng.choice(["none", "none", "fp32", "same"])
        if case["base"] != "none":  # read as well as written
            case["vocab"] = max(1, vocab // 3)
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


def _tokens(n, vocab, gen, dev):
    """Tokens as text has them: the k-th most frequent one about 1/k as often as the first."""
    weight = 1.0 / (torch.arange(vocab, dtype=torch.float64, device=dev) + 2.7)
    upto = torch.cumsum(weight, 0)
    u = torch.rand(n, generator=gen, device=dev, dtype=torch.float64) * upto[-1]
    rank = torch.searchsorted(upto, u).clamp_max(vocab - 1)
    return torch.randperm(vocab, generator=gen, device=dev)[rank]


CLIP_LOW, CLIP_HIGH = 0.2, 0.28


def _prepare_policy(case, gen, dev):
    rows, vocab, c = case["rows"], case["vocab"], case["scale"]
    x = _logits(case, gen, dev)
    # most sampled tokens are likely ones; every seventh row has any token
    likely = x[:, :min(vocab, 4096)].argmax(dim=1)
    anyone = torch.randint(0, vocab, (rows,), generator=gen, device=dev)
    tokens = torch.where(torch.arange(rows, device=dev) % 7 == 3, anyone, likely)
    lp = torch.empty(rows, dtype=torch.float64, device=dev)
    step = max(1, (1 << 26) // vocab)
    for r in range(0, rows, step):
        z = x[r:r + step].double() * c
        lp[r:r + step] = z.gather(1, tokens[r:r + step, None])[:, 0] - torch.logsumexp(z, dim=1)
    # the log ratios of a policy a few updates old. The gradient jumps at the borders of the clipping: no ratio is put so
    # near one that the rounding of its log probability to 32 bits says on which side it is
    ratio = 0.15 * torch.randn(rows, generator=gen, device=dev, dtype=torch.float64)
    for border in (1.0 - CLIP_LOW, 1.0 + CLIP_HIGH, 3.0):
        ratio = torch.where((ratio - math.log(border)).abs() < 1e-4, ratio + 3e-4, ratio)
    f32 = dict(dtype=torch.float32, device=dev)
    s = {"x": x, "tokens": tokens.to(IDTYPES[case["ids"]]), "old": (lp - ratio).float() if case["old"] else None,
         "advantage": torch.randn(rows, generator=gen, **f32), "ref": None, "weight": None}
    if case["kl"] != "none":
        s["ref"] = (lp + 0.3 * torch.randn(rows, generator=gen, device=dev, dtype=torch.float64)).float()
    if case["skip"]:  # prompt positions, which carry nothing
        s["weight"] = torch.full((rows,), 1.0 / rows, **f32)
        s["weight"][case["skip"] - 1::case["skip"]] = 0.0
    s["out"] = {k: torch.empty(rows, **f32) for k in ("loss", "ratio")}
    if s["ref"] is not None:
        s["out"]["kl"] = torch.empty(rows, **f32)
    if case["op"] == "policy":
        s["d_logits"] = torch.empty((rows, vocab + case["pad"]), dtype=x.dtype, device=dev)[:, :vocab]
    else:
        s["out"].update({k: torch.empty(rows, **f32) for k in ("logprob", "entropy", "d_logprob", "d_entropy")})
        s["out"]["norm"] = torch.empty((rows, 2), **f32)
    return s


def _prepare_preference(case, gen, dev):
    pairs, tokens = case["pairs"], case["tokens"]
    rows = tokens + case["behind"]
    # answers of uneven lengths that fill the tokens, rows behind the last of them
    ends = torch.cumsum(torch.rand(2 * pairs, generator=gen, device=dev, dtype=torch.float64) + 0.2, 0)
    offsets = torch.zeros(2 * pairs + 1, dtype=torch.int64, device=dev)
    offsets[1:] = (ends / ends[-1] * tokens).round().long()
    f32 = dict(dtype=torch.float32, device=dev)
    lp = -2.0 * torch.empty(rows, **f32).exponential_(1.0, generator=gen)
    at = torch.arange(rows, device=dev)
    seq = torch.searchsorted(offsets, at, right=True) - 1
    first = offsets[seq.clamp_max(2 * pairs)]
    weight = (at - first >= 5).float()  # the last tokens of the prompt, which both answers have
    return {"logprob": lp, "ref": lp + 0.1 * torch.randn(rows, generator=gen, **f32) if case["ref"] else None,
            "weight": weight, "offsets": offsets.to(IDTYPES[case["ids"]]), "beta": 0.125 if case["ref"] else 2.0,
            "margin": 0.0 if case["ref"] else 0.5,
            "out": {"loss": torch.empty(pairs, **f32), "reward": torch.empty((pairs, 2), **f32),
                    "d_logprob": torch.zeros(rows, **f32)}}


def _prepare_embedding(case, gen, dev):
    n, vocab, dim = case["n"], case["vocab"], case["dim"]
    ids = _tokens(n, vocab, gen, dev)
    if case["holes"]:
        ids[case["holes"] - 1::case["holes"]] = -1  # padding
    s = {"ids": ids.to(IDTYPES[case["ids"]])}
    if case["op"] == "embedding":
        s["table"] = (torch.randn((vocab, dim), generator=gen, device=dev) * 0.02).to(DTYPES[case["dtype"]])
        s["out"] = torch.empty((n, dim), dtype=DTYPES[case["out"]], device=dev)
        return s
    s["d_out"] = (torch.randn((n, dim), generator=gen, device=dev) * 0.01).to(DTYPES[case["dtype"]])
    s["d_table"] = torch.empty((vocab, dim), dtype=DTYPES[case["out"]], device=dev)
    s["base"] = None
    if case["base"] != "none":
        s["base"] = torch.randn((vocab, dim), generator=gen, device=dev) * 0.01
        if case["base"] == "same":
            s["base"] = s["base"].to(DTYPES[case["out"]])
    return s


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    make = {"poli": _prepare_policy, "pref": _prepare_preference, "embe": _prepare_embedding}[case["op"][:4]]
    return {"case": case, **make(case, gen, dev)}


# ------------------------------------------------------------------ the plain form

def _plain_policy(s):
    x, case = s["x"], s["case"]
    c, adv, tok = case["scale"], s["advantage"], s["tokens"].long()[:, None]
    top = x.max(dim=1, keepdim=True).values.float()
    d = (x.float() - top) * c
    e = torch.exp(d)
    t = e.sum(dim=1, keepdim=True)
    log_t = torch.log(t)
    w = s["weight"] if s["weight"] is not None else torch.ones_like(adv)
    live = w != 0
    # the ratios in 64 bits: the clipping has borders
    lp = d.gather(1, tok)[:, 0].double() - torch.log(t.double())[:, 0]
    ratio = torch.exp(lp - s["old"]) if s["old"] is not None else torch.ones_like(lp)
    up = adv >= 0
    low = torch.where(up, 0.0, 1.0 - CLIP_LOW)
    high = torch.where(up, 1.0 + CLIP_HIGH, case["dual"] if case["dual"] else math.inf)
    loss = -adv * torch.minimum(torch.maximum(ratio, low), high)
    d_lp = torch.where((ratio >= low) & (ratio <= high), -adv * ratio, 0.0)
    out = {"ratio": torch.where(live, ratio, 0.0).float()}
    if s["ref"] is not None:
        gap = lp - s["ref"]
        kl = {"k1": gap, "k2": 0.5 * gap * gap, "k3": torch.exp(-gap) + gap - 1.0}[case["kl"]]
        d_kl = {"k1": torch.ones_like(gap), "k2": gap, "k3": 1.0 - torch.exp(-gap)}[case["kl"]]
        loss = loss + case["kl_coef"] * kl
        d_lp = d_lp + case["kl_coef"] * d_kl
        out["kl"] = torch.where(live, kl, 0.0).float()
    entropy = log_t[:, 0] - (e * d).sum(dim=1) / t[:, 0]
    loss = loss - case["entropy"] * entropy
    d_lp = torch.where(live, d_lp * w, 0.0).float()
    d_h = torch.where(live, -case["entropy"] * w, 0.0)
    out["loss"] = torch.where(live, loss * w, 0.0).float()
    if case["op"] == "policy_loss":
        out.update(logprob=torch.where(live, lp, 0.0).float(), entropy=torch.where(live, entropy, 0.0), d_logprob=d_lp,
                   d_entropy=d_h, norm=torch.where(live[:, None], torch.cat([top, t], dim=1), 0.0))
        return out
    p = e / t
    g = -p * d_lp[:, None]
    if case["entropy"]:
        g = g - d_h[:, None] * p * (d - log_t + entropy[:, None])
    g.scatter_add_(1, tok, d_lp[:, None])
    out["d_logits"] = (g * c).to(x.dtype)
    return out


def _plain_preference(s):
    case, lp, w = s["case"], s["logprob"], s["weight"]
    pairs = case["pairs"]
    offsets = s["offsets"].long()
    at = torch.arange(lp.numel(), device=lp.device)
    seq = torch.searchsorted(offsets, at, right=True) - 1  # rows behind the last sequence: 2 * pairs
    lr = lp - s["ref"] if s["ref"] is not None else lp
    f64 = dict(dtype=torch.float64, device=lp.device)
    total = torch.zeros(2 * pairs + 1, **f64).index_add_(0, seq, (w * lr).double())[:2 * pairs]
    count = torch.zeros(2 * pairs + 1, **f64).index_add_(0, seq, w.double())[:2 * pairs]
    per = torch.where(count > 0, 1.0 / count, 0.0) if case["average"] else torch.ones_like(count)
    score = (total * per).view((2, pairs) if case["halves"] else (pairs, 2))
    chosen, rejected = (score[0], score[1]) if case["halves"] else (score[:, 0], score[:, 1])
    beta, eps = s["beta"], case["smooth"]
    h = beta * (chosen - rejected) - s["margin"]
    if case["kind"] == "sigmoid":
        soft = torch.log1p(torch.exp(-h.abs()))
        loss = (1 - eps) * ((-h).clamp_min(0) + soft) + eps * (h.clamp_min(0) + soft)
        d_h = 1.0 / (1.0 + torch.exp(-h)) - (1 - eps)
    elif case["kind"] == "hinge":
        loss = (1.0 - h).clamp_min(0)
        d_h = -(h < 1.0).double()
    else:
        loss = ((h - 0.5) / beta) ** 2
        d_h = 2.0 * (h - 0.5) / beta ** 2
    d_score = torch.stack([d_h * beta, -d_h * beta], dim=0 if case["halves"] else 1).reshape(-1) * per
    d_score = torch.cat([d_score, torch.zeros(1, **f64)])
    return {"loss": loss.float(), "reward": (beta * torch.stack([chosen, rejected], dim=1)).float(),
            "d_logprob": (d_score[seq] * w).float()}


def _plain_embedding(s):
    case, ids = s["case"], s["ids"].long()
    there = (ids >= 0)[:, None]
    if case["op"] == "embedding":
        rows = s["table"][ids.clamp_min(0)].float() * case["scale"]
        return torch.where(there, rows, 0.0).to(DTYPES[case["out"]])
    g = torch.where(there, s["d_out"].float(), 0.0)
    total = torch.zeros((case["vocab"], case["dim"]), device=g.device).index_add_(0, ids.clamp_min(0), g)
    total = total * case["scale"]
    if s["base"] is not None:
        total = total + s["base"].float()
    return total.to(DTYPES[case["out"]])


# ------------------------------------------------------------------ one pass

def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return (_plain_policy if op.startswith("policy") else
                _plain_preference if op == "preference" else _plain_embedding)(s)
    import fsdp_sharded_mixed_ss_gb300 as ss

    if op.startswith("policy"):
        kl = {"none": ss.SS_KL_K3, "k1": ss.SS_KL_K1, "k2": ss.SS_KL_K2, "k3": ss.SS_KL_K3}[case["kl"]]
        ss.ss_policy_loss(s["x"], s["tokens"], s["advantage"], old_logprob=s["old"], ref_logprob=s["ref"],
                          row_weight=s["weight"], clip_low=CLIP_LOW, clip_high=CLIP_HIGH, clip_max=case["dual"], kl_kind=kl,
                          kl_coef=case["kl_coef"], entropy_coef=case["entropy"], scale=case["scale"],
                          d_logits=s.get("d_logits"), **s["out"])
        return {**s["out"], "d_logits": s["d_logits"]} if op == "policy" else s["out"]
    if op == "preference":
        kind = {"sigmoid": ss.SS_PREF_SIGMOID, "hinge": ss.SS_PREF_HINGE, "square": ss.SS_PREF_SQUARE}[case["kind"]]
        ss.ss_preference_loss(s["logprob"], s["offsets"], ref_logprob=s["ref"], row_weight=s["weight"], kind=kind,
                              beta=s["beta"], margin=s["margin"], label_smoothing=case["smooth"],
                              average=case["average"], halves=case["halves"], **s["out"])
        return s["out"]
    if op == "embedding":
        ss.ss_embedding(s["table"], s["ids"], s["out"], scale=case["scale"])
        return s["out"]
    if "workspace" not in s:
        s["workspace"] = torch.empty(ss.ss_embedding_grad_workspace(case["n"], case["vocab"], case["dim"]),
                                     dtype=torch.uint8, device=s["ids"].device)
    ss.ss_embedding_grad(s["d_out"], s["ids"], s["d_table"], s["workspace"], base=s["base"], scale=case["scale"])
    return s["d_table"]


def _distinct(n, vocab):
    """Tokens that n draws are expected to name."""
    weight = 1.0 / (torch.arange(vocab, dtype=torch.float64) + 2.7)
    return int(-torch.expm1(n * torch.log1p(-weight / weight.sum())).sum())


def work(case):
    """Each input once and each output once. A position that carries nothing is not read; its gradient is written."""
    op, ib = case["op"], BYTES[case["ids"]]
    if op.startswith("policy"):
        rows, es = case["rows"], BYTES[case["dtype"]]
        n = rows * case["vocab"]
        live = rows - rows // case["skip"] if case["skip"] else rows
        read = live * case["vocab"]
        small = rows * (ib + 16 + 4 * case["old"] + 8 * (case["kl"] != "none"))
        if op == "policy_loss":
            return {"bytes": read * es + small + rows * 24, "flops": 6 * read}
        return {"bytes": (read + n) * es + small, "flops": 11 * read}
    if op == "preference":
        return {"bytes": case["tokens"] * (16 if case["ref"] else 12) + case["pairs"] * (2 * ib + 12),
                "flops": 5 * case["tokens"]}
    n, dim = case["n"], case["dim"]
    live = n - n // case["holes"] if case["holes"] else n
    if op == "embedding":
        read = _distinct(live, case["vocab"]) * dim * BYTES[case["dtype"]]
        return {"bytes": read + n * (ib + dim * BYTES[case["out"]]), "flops": live * dim}
    table = case["vocab"] * dim
    base = {"none": 0, "fp32": 4, "same": BYTES[case["out"]]}[case["base"]]
    return {"bytes": n * ib + live * dim * BYTES[case["dtype"]] + table * (BYTES[case["out"]] + base),
            "flops": live * dim + table}


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_policy(s):
    """The loss as the minimum of two products, its gradient by differentiating it."""
    case, parts = s["case"], []
    rows = case["rows"]
    weight = s["weight"] if s["weight"] is not None else torch.ones(rows, device=s["x"].device)
    step = max(1, (1 << 24) // case["vocab"])
    for r in range(0, rows, step):
        sl = slice(r, min(rows, r + step))
        x = s["x"][sl].double()
        z = x.clone().requires_grad_(True)
        logp = torch.log_softmax(z * case["scale"], dim=1)
        lp = logp.gather(1, s["tokens"][sl].long()[:, None])[:, 0]
        entropy = -(logp.exp() * logp).sum(dim=1)
        adv, w = s["advantage"][sl].double(), weight[sl].double()
        old = s["old"][sl].double() if s["old"] is not None else lp.detach()
        ratio = (lp - old).exp()
        gain = torch.minimum(ratio * adv, ratio.clamp(1.0 - CLIP_LOW, 1.0 + CLIP_HIGH) * adv)
        if case["dual"]:
            gain = torch.where(adv < 0, torch.maximum(gain, case["dual"] * adv), gain)
        loss = -gain - case["entropy"] * entropy
        o = {"ratio": ratio}
        if s["ref"] is not None:
            back = s["ref"][sl].double() - lp
            o["kl"] = {"k1": -back, "k2": back.square() / 2, "k3": torch.expm1(back) - back}[case["kl"]]
            loss = loss + case["kl_coef"] * o["kl"]
        loss = loss * w
        d_lp, d_h, d_x = torch.autograd.grad(loss.sum(), (lp, entropy, z), allow_unused=True)
        o["loss"] = loss
        o = {k: torch.where(w != 0, v.detach(), 0.0) for k, v in o.items()}
        if case["op"] == "policy":
            o["d_logits"] = d_x
        else:
            big = x.max(dim=1).values
            sums = ((x - big[:, None]) * case["scale"]).exp().sum(dim=1)
            dead = w == 0
            o.update(logprob=lp.detach().masked_fill(dead, 0.0), entropy=entropy.detach().masked_fill(dead, 0.0),
                     d_logprob=d_lp, d_entropy=d_h, norm=torch.stack([big, sums], dim=1).masked_fill(dead[:, None], 0.0))
        parts.append(o)
    return {k: torch.cat([o[k] for o in parts]) for k in parts[0]}


def _exact_preference(s):
    """The sums of single sequences as differences of running sums, the loss's derivatives by differentiating it."""
    case = s["case"]
    lr = s["logprob"].double()
    if s["ref"] is not None:
        lr = lr - s["ref"].double()
    w = s["weight"].double()
    o = s["offsets"].long()
    zero = torch.zeros(1, dtype=torch.float64, device=lr.device)
    total = torch.cat([zero, torch.cumsum(lr * w, 0)])[o].diff()
    count = torch.cat([zero, torch.cumsum(w, 0)])[o].diff()
    if case["average"]:
        total = total / count.clamp_min(1.0)
    score = (total.view(2, -1).t() if case["halves"] else total.view(-1, 2)).clone().requires_grad_(True)
    h = s["beta"] * (score[:, 0] - score[:, 1]) - s["margin"]
    soft = torch.nn.functional.softplus
    eps = case["smooth"]
    loss = {"sigmoid": lambda: (1 - eps) * soft(-h, threshold=1e9) + eps * soft(h, threshold=1e9),
            "hinge": lambda: torch.relu(1.0 - h),
            "square": lambda: ((h - 0.5) / s["beta"]).square()}[case["kind"]]()
    g, = torch.autograd.grad(loss.sum(), score)
    g = (g.t() if case["halves"] else g).reshape(-1)
    if case["average"]:
        g = g / count.clamp_min(1.0)
    d = torch.zeros_like(lr)
    d[int(o[0]):int(o[-1])] = torch.repeat_interleave(g, o.diff())
    return {"loss": loss.detach(), "reward": (score * s["beta"]).detach(), "d_logprob": d * w}


def _exact_embedding(s):
    """The lookup row by row; the gradient as differences of running sums over the positions in order of their tokens."""
    case = s["case"]
    ids = s["ids"].long()
    live = torch.nonzero(ids >= 0)[:, 0]
    if case["op"] == "embedding":
        out = torch.zeros((case["n"], case["dim"]), dtype=torch.float64, device=ids.device)
        out[live] = torch.index_select(s["table"], 0, ids[live]).double() * case["scale"]
        return out
    key, order = torch.sort(ids[live], stable=True)
    order = live[order]
    name, count = torch.unique_consecutive(key, return_counts=True)
    last = torch.cumsum(count, 0) - 1
    out = torch.zeros((case["vocab"], case["dim"]), dtype=torch.float64, device=ids.device)
    for c in range(0, case["dim"], 512):
        if name.numel():
            upto = torch.cumsum(s["d_out"][order, c:c + 512].double(), 0)[last]
            out[name, c:c + 512] = torch.diff(upto, dim=0, prepend=torch.zeros_like(upto[:1])) * case["scale"]
        if s["base"] is not None:
            out[:, c:c + 512] += s["base"][:, c:c + 512].double()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"poli": _exact_policy, "pref": _exact_preference, "embe": _exact_embedding}[case["op"][:4]](s)
