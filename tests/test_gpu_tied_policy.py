"""The losses on sampled tokens and the embedding together, as a training step uses them: the example runs, one rank's table
gradient against float64 and against differences of the loss, and a step captured into a graph beside eager calls."""
import importlib.util
import os

import numpy as np
import pytest

from policy_ref import row_policy

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("tied_policy", os.path.join(ROOT, "examples", "tied_policy.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _batch(rows, vocab, seed=0):
    rng = np.random.default_rng(seed)
    f = lambda a: torch.tensor(a, dtype=torch.float32, device="cuda")  # noqa: E731
    previous = torch.tensor(rng.integers(0, vocab // 4, rows), device="cuda")   # tokens that occur again and again
    previous[3] = -1
    w = rng.uniform(0.5, 1.5, rows) / rows
    w[5] = 0.0
    return previous, dict(tokens=torch.tensor(rng.integers(0, vocab, rows), device="cuda"), advantage=f(rng.normal(size=rows)),
                          weight=f(w))


def _setup(ss, example, dtype, rows=70, vocab=301, dim=48):
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    table = (torch.randn((vocab, dim), generator=g, device="cuda") * 0.3).to(dtype)
    previous, b = _batch(rows, vocab)
    lp = example.log_probs(table, previous, b["tokens"], 2.0)
    b["old"], b["reference"] = lp - 0.05, lp + 0.3
    ws = torch.empty(ss.ss_embedding_grad_workspace(rows, vocab, dim), dtype=torch.uint8, device="cuda")
    return table, previous, b, ws


def test_example_runs(example):
    rewards = example.train(rounds=3, updates=2, vocab=503, dim=32, rows=96, n_ranks=3)
    assert len(rewards) == 3 and all(0.0 <= r <= 1.0 for r in rewards)


def test_table_gradient_against_float64(example):
    """fp32 tables, so that only the calls' own roundings count beside the products'."""
    import fsdp_sharded_mixed_ss_gb300 as ss

    torch.backends.cuda.matmul.allow_tf32 = False
    table, previous, b, ws = _setup(ss, example, torch.float32)
    scale = 2.0
    loss, got = example.table_gradient(table, previous, b, scale, ws, kl_coef=0.2, entropy_coef=0.05)
    torch.cuda.synchronize()
    T = table.double().cpu().numpy()
    P, K = previous.cpu().numpy(), b["tokens"].cpu().numpy()
    H = np.where((P >= 0)[:, None], T[np.maximum(P, 0)], 0.0) * scale
    X = H @ T.T
    f32 = lambda v: float(np.float32(v))  # noqa: E731
    D, L = np.zeros_like(X), np.zeros(len(P))
    for r in range(len(P)):
        o, _, g, _ = row_policy(X[r], 1.0, int(K[r]), float(b["advantage"][r]), old=float(b["old"][r]),
                                ref=float(b["reference"][r]), weight=float(b["weight"][r]), kind="k3", kc=f32(0.2),
                                ec=f32(0.05), low=f32(0.2), high=f32(0.2))
        D[r], L[r] = g, o["loss"]
    want = D.T @ H
    dH = (D @ T) * scale
    np.add.at(want, P[P >= 0], dH[P >= 0])
    # the logits are products of 48 terms in fp32, 48 * 2^-24 of values whose absolute sum is below 60 (48 terms of 0.09 by
    # 2, a few times over): below 2e-4, and the rows' derivatives are that smooth; REL on the rows beside it
    size = np.abs(D).T @ np.abs(H)
    np.add.at(size, P[P >= 0], (np.abs(D) @ np.abs(T) * scale)[P >= 0])
    err = np.abs(got.double().cpu().numpy().reshape(want.shape) - want)
    assert (err <= 1e-3 * size + 1e-3 * size.mean()).all(), float((err / (size + size.mean())).max())
    assert (np.abs(loss.double().cpu().numpy() - L) <= 1e-3 * (np.abs(L) + 1.0 / len(P))).all()


def test_table_gradient_against_differences(example):
    import fsdp_sharded_mixed_ss_gb300 as ss

    torch.backends.cuda.matmul.allow_tf32 = False
    table, previous, b, ws = _setup(ss, example, torch.float32)
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    v = torch.randn(table.shape, generator=g, device="cuda")
    h = 2.0 ** -9
    kw = dict(kl_coef=0.2, entropy_coef=0.05)
    _, d = example.table_gradient(table, previous, b, 2.0, ws, **kw)
    plus, _ = example.table_gradient(table + h * v, previous, b, 2.0, ws, **kw)
    minus, _ = example.table_gradient(table - h * v, previous, b, 2.0, ws, **kw)
    slope = float((plus.double() - minus.double()).sum()) / (2 * h)
    got = float((d.double() * v.reshape(-1).double()).sum())
    # ratios stay near 1.05, off the borders. The losses' errors, 2e-4 of a few tenths, fall over the step and the rows
    # (their mean); the third derivative along v, of logits that move by about 7 and are quadratic, is below 2000
    assert abs(got - slope) <= 2e-4 / h / np.sqrt(len(previous)) + h * h * 2000 / 6, (got, slope)


def test_step_captured_beside_eager_calls(example):
    """A rank's whole gradient in a graph, replayed with eager calls on other data in between."""
    import fsdp_sharded_mixed_ss_gb300 as ss

    table, previous, b, ws = _setup(ss, example, torch.bfloat16)
    want_loss, want = example.table_gradient(table, previous, b, 2.0, ws)
    other = _setup(ss, example, torch.bfloat16, rows=33, vocab=120)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, d = example.table_gradient(table, previous, b, 2.0, ws)
    for _ in range(3):
        example.table_gradient(*other[:3], 2.0, other[3])
        loss.zero_()
        d.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(loss, want_loss) and torch.equal(d, want)


def test_gradient_goes_through_the_shard_step(example):
    """The 16-bit gradients of two ranks, summed and stepped by the fused kernel of every shard, against torch in float64."""
    import fsdp_sharded_mixed_ss_gb300 as ss

    policy = example.Head(301, 48, 2, "cuda", seed=3)
    table = policy.weight.clone()
    grads = []
    for seed in (1, 2):
        previous, b = _batch(70, 301, seed)
        b["old"] = example.log_probs(table, previous, b["tokens"], 2.0)
        b["reference"] = b["old"] + 0.2
        ws = torch.empty(ss.ss_embedding_grad_workspace(70, 301, 48), dtype=torch.uint8, device="cuda")
        grads.append(example.table_gradient(table, previous, b, 2.0, ws)[1])
    before = torch.cat(policy.master).double()
    policy.step(grads, 1, 1e-2, max_norm=1e9)
    torch.cuda.synchronize()
    g = (grads[0].double() + grads[1].double()) / 2
    want = before - 1e-2 * g / (g.abs() + 1e-8)       # AdamW's first step
    got = torch.cat(policy.master).double()
    # the mean gradient rounds to fp32, and the hyperparameters are fp32
    assert bool(((got - want).abs() <= 1e-6 * want.abs() + 1e-2 * 1e-6).all())
    assert torch.equal(policy.flat, got.float().to(torch.bfloat16))
