"""Sampling in its largest forms: clusters of 2 to 8 CTAs over long rows, the longest row, more rows than are sorted."""
import numpy as np
import pytest

from gpu_util import require_gpu

pytestmark = pytest.mark.gpu

# Weights are formed to 2^-29 of themselves and summed exactly, the reference's sums in float64 (2^18 additions of 2^-53):
# a border between two tokens lies within 2^-28 of the total of where the definition has it.
EPS = 2.0 ** -28


@pytest.fixture(scope="module")
def torch():
    return require_gpu()


@pytest.fixture(scope="module")
def F(torch):
    from tree_forked_hybrid_gb300 import fork
    return fork


def run(F, torch, x, u, **par):
    rows = x.shape[0]
    dt = {"top_k": torch.int32}
    dev = {k: torch.from_numpy(np.asarray(v)).to(dt.get(k, torch.float32)).cuda() for k, v in par.items()}
    token = torch.full((rows,), -9, dtype=torch.int32, device="cuda")
    prob = torch.full((rows,), -9.0, device="cuda")
    F.fork_sample(x, token, torch.from_numpy(np.asarray(u, np.float32)).cuda(), prob=prob, **dev)
    return token, prob


def kept_weights(torch, x, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """float64 weights of one row with what is cut set to zero, and how far the cuts of top-p and min-p are from a border."""
    x = x.double()
    w = torch.exp((x - x.max()) / temperature)
    order = torch.sort(x, descending=True, stable=True).indices
    ws = w[order]
    keep = torch.ones_like(ws, dtype=torch.bool)
    clear = float("inf")
    if top_k > 0:
        keep[top_k:] = False
    ws = ws * keep
    if top_p < 1:
        before = torch.cumsum(ws, 0) - ws
        share = top_p * ws.sum()
        clear = float(((before - share).abs() / ws.sum())[ws > 0].min())
        keep &= before < share
    if min_p > 0:
        clear = min(clear, float((ws / min_p - 1).abs().min()))
        keep &= ws >= min_p
    keep[0] = True
    out = torch.zeros_like(w)
    out[order] = ws * keep
    return out, clear


def check(F, torch, x, u, only=None, **par):
    token, prob = run(F, torch, x, u, **par)
    token, prob = token.tolist(), prob.tolist()
    for r in range(x.shape[0]) if only is None else only:
        one = {k: np.asarray(v, {"top_k": np.int32}.get(k, np.float32))[r].item() for k, v in par.items()}
        w, clear = kept_weights(torch, x[r].float(), **one)
        if clear <= EPS:  # (a cut that rounding may move by a token says nothing here)
            continue
        run_sum = torch.cumsum(w, 0)
        total = float(run_sum[-1])
        t = token[r]
        assert 0 <= t < x.shape[1] and float(w[t]) > 0, (r, one, t)
        at = np.float32(u[r]).item() * total
        assert float(run_sum[t]) - float(w[t]) - EPS * total <= at <= float(run_sum[t]) + EPS * total, (r, one, t)
        want = float(w[t]) / total
        assert abs(prob[r] - want) <= want * (2.0 ** -24 + EPS), (r, one, prob[r], want)


KINDS = [dict(), dict(top_k=50), dict(top_k=3000), dict(top_p=0.9), dict(top_p=0.999), dict(min_p=0.01), dict(min_p=1e-6),
         dict(top_k=100, top_p=0.8), dict(top_k=40000, top_p=0.95, min_p=1e-5)]


@pytest.mark.parametrize("k", range(len(KINDS)))
@pytest.mark.parametrize("rows,V", [(1, 131072), (5, 131071), (19, 131072), (1, 1 << 18), (5, (1 << 18) - 5), (19, 1 << 18),
                                    (40, 1 << 18), (160, 1 << 18)])
@pytest.mark.parametrize("bf16", [False, True])
def test_long_rows(F, torch, k, rows, V, bf16):
    """Rows of several spreads, at every alignment that an odd stride and base give."""
    g = torch.Generator(device="cuda").manual_seed(100 * k + rows)
    wide = torch.zeros((rows, V + 3), device="cuda", dtype=torch.bfloat16 if bf16 else torch.float32)
    x = wide[:, 1:1 + V]
    v = torch.randn((rows, V), device="cuda", generator=g) * torch.linspace(0.3, 4, rows, device="cuda")[:, None]
    at = torch.randint(0, V, (rows, 20), device="cuda", generator=g)
    v.scatter_add_(1, at, torch.rand((rows, 20), device="cuda", generator=g) * 12)
    x.copy_(v)
    rng = np.random.default_rng(k)
    par = {n: np.full(rows, p) for n, p in KINDS[k].items()}
    check(F, torch, x, rng.random(rows), temperature=rng.uniform(0.4, 1.5, rows), only=range(0, rows, max(1, rows // 6)), **par)


@pytest.mark.parametrize("rows", [1, 5, 19, 160])
def test_flat_rows_of_the_longest_kind(F, torch, rows):
    """2^18 equal weights: the largest sums there are; every border is known exactly."""
    V = 1 << 18
    x = torch.full((rows, V), 3.5, device="cuda")
    i = np.linspace(0, V - 1, rows).astype(np.int64)
    u = ((i + 0.5) / V).astype(np.float32)
    token, prob = run(F, torch, x, u)
    assert token.tolist() == i.tolist() and prob.tolist() == [2.0 ** -18] * rows
    token, prob = run(F, torch, x, u, top_p=np.full(rows, 0.5))
    assert token.tolist() == (i // 2).tolist() and prob.tolist() == [2.0 ** -17] * rows
    token, _ = run(F, torch, x, u, top_k=np.full(rows, V // 4))
    assert token.tolist() == (i // 4).tolist()
    token, _ = run(F, torch, x, np.full(rows, 1 - 2.0 ** -24), temperature=np.full(rows, 0.01), min_p=np.full(rows, 1.0))
    assert token.tolist() == [V - 1] * rows


@pytest.mark.parametrize("rows", [1, 19, 160])
@pytest.mark.parametrize("octaves", [5.0, 5.3, 9.9, 10.1, 13.0, 23.9, 24.1])
def test_nearly_all_tokens_far_below_the_largest(F, torch, rows, octaves):
    """Some 2^18 light tokens in one or a few bins, top-p close to 1: counts and sums of the bins at their largest."""
    V = 1 << 18
    g = torch.Generator(device="cuda").manual_seed(rows)
    one = -octaves * np.log(2.0) + 0.01 * torch.randn(V, device="cuda", generator=g)
    one[torch.randint(0, V, (3,), device="cuda", generator=g)] = 0.0
    x = one[None].repeat(rows, 1)
    p = 1 - np.geomspace(0.3, 1e-5, rows)
    u = np.random.default_rng(rows).random(rows)
    check(F, torch, x, u, top_p=p, only=range(0, rows, max(1, rows // 8)))
    x[:, ::2] = -octaves * np.log(2.0)  # half of them equal
    check(F, torch, x, u, top_p=p, only=range(0, rows, max(1, rows // 8)))


def test_more_rows_than_are_sorted(F, torch):
    rows, V = 4097, 513
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn((rows, V), device="cuda", generator=g) * 3
    rng = np.random.default_rng(0)
    kind = np.arange(rows) % 4
    check(F, torch, x, rng.random(rows), only=[*range(0, rows, 37), rows - 1], temperature=rng.uniform(0.3, 1.5, rows),
          top_k=np.where(kind == 1, 20, 0), top_p=np.where(kind == 2, 0.9, 1.0), min_p=np.where(kind == 3, 0.02, 0.0))
