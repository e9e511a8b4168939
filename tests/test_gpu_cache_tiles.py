"""Every tile of a long context counts once: zero queries weigh all seen keys alike, and values mark their tile."""
import numpy as np
import pytest

from cache_util import make_step
from gpu_util import require_gpu
from test_gpu_cache_attn import reference, run

pytestmark = pytest.mark.gpu

TILE = 128


@pytest.fixture(scope="module")
def torch():
    return require_gpu()


@pytest.fixture(scope="module")
def F(torch):
    from tree_forked_hybrid_gb300 import fork
    return fork


def marked(torch, st, Hkv, d):
    """Keys of noise; values of tile t: 2^(t // d) in column t % d, and -2^(t // d) in the next column of the next kv
    head, zeros elsewhere.  Sums over whole tiles are integers below 2^24: exact in float32 in any order."""
    g = torch.Generator(device="cuda").manual_seed(1)
    kc = torch.randn((st["n_pages"], Hkv, st["page"], d), device="cuda", generator=g).to(torch.bfloat16)
    vc = torch.zeros_like(kc)
    P = st["page"]
    for b, (ln, n) in enumerate(zip(st["length"], np.maximum(st["n_new"], 0))):
        y = np.arange(int(ln + n))
        page = torch.from_numpy(st["table"][b, y // P].astype(np.int64)).cuda()
        off, t = torch.from_numpy(y % P).cuda(), y // TILE
        mark = torch.from_numpy(2.0 ** (t // d)).cuda().to(torch.bfloat16)
        for h in range(Hkv):
            col = torch.from_numpy((t + h) % d).cuda()
            vc[page, h, off, col] = mark if h % 2 == 0 else -mark
    return kc, vc


# small kernel: 16 rows (heads of 64 and 128) and 32; tcgen05: one query tile and two
FORMS = [(4, 1, 128, 1, False), (8, 4, 64, 2, True), (8, 1, 64, 4, True), (16, 2, 128, 9, True), (16, 4, 64, 30, True),
         (16, 2, 128, 40, True), (32, 1, 64, 9, False), (12, 3, 128, 70, False)]


@pytest.mark.parametrize("k", range(len(FORMS)))
@pytest.mark.parametrize("lengths,page", [
    ([30700], 128),                      # one request, 240 tiles and a new one's: with one kv head 152 pieces to join
    ([12799, 128 * 90, 11000, 5], 64),   # items of 85 to 100 tiles beside one another
    ([2000] * 40, 16)])                  # many items of 16 tiles
@pytest.mark.parametrize("window", [0, 1000, 10241])
def test_every_tile_counts_once(F, torch, k, lengths, page, window):
    """Weights are 1, products with the marks and sums exact: what is left is 1 / sum (a few roundings of 2^-24) and the
    rounding of the result, 2^-8.  A column has at most four marks, of 1, 2, 4 and 8: a tile left out or taken twice
    moves its own by 1 part in 15 or more."""
    Hq, Hkv, d, n, tree = FORMS[k]
    st = make_step(17 + k, lengths, [n] * len(lengths), page, tree)
    kc, vc = marked(torch, st, Hkv, d)
    q = torch.zeros((st["T_cap"], Hq, d), dtype=torch.bfloat16, device="cuda")
    got, _ = run(F, torch, st, q, kc, vc, Hq, Hkv, d, window)
    want, _ = reference(torch, st, q, kc, vc, window, d ** -0.5)
    err = (got.double() - want).abs()
    assert bool((err <= want.abs() * (2.0 ** -8 + 2.0 ** -20)).all()), float((err / (want.abs() + 1e-30)).max())


@pytest.mark.parametrize("k", range(len(FORMS)))
def test_one_key_carries_each_row(F, torch, k):
    """A query meets one key, the first, a middle or the last one of a tile, with a score 100 above all others: the result
    is that key's value, wherever runs begin and end."""
    Hq, Hkv, d, n, tree = FORMS[k]
    G = Hq // Hkv
    g = torch.Generator(device="cuda").manual_seed(k)
    st = make_step(3, [30011, 9000], [n, n], 32, tree)
    kc = torch.zeros((st["n_pages"], Hkv, 32, d), dtype=torch.bfloat16, device="cuda")
    vc = torch.randn(kc.shape, device="cuda", generator=g).to(torch.bfloat16)
    tiles = np.arange(30011 // TILE)
    for first in range(0, len(tiles) * 3, d // 2):  # a group of keys at a time, a dimension each
        kc.zero_()
        at = [(t * TILE + o) for t in tiles for o in (0, 63, 127)][first:first + d // 2]
        y = torch.tensor(at, device="cuda")
        page = torch.from_numpy(st["table"][0].astype(np.int64)).cuda()[y // 32]
        dim = torch.arange(len(at), device="cuda")
        for h in range(Hkv):
            kc[page, h, y % 32, dim] = 100.0
        q = torch.zeros((st["T_cap"], Hq, d), dtype=torch.bfloat16, device="cuda")
        rows = torch.arange(n * Hq, device="cuda")
        pick = (rows * 7 + first) % len(at)
        q[:n].view(n * Hq, d)[rows, pick] = 1.0
        got, _ = run(F, torch, st, q, kc, vc, Hq, Hkv, d, 0, 1.0)
        # (the others together weigh 30011 e^-100)
        head = rows % Hq // G
        assert torch.equal(got[:n].reshape(n * Hq, d), vc[page[pick], head, y[pick] % 32])
