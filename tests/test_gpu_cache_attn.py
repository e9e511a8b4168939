"""Attention over the paged cache on the GPU against the float64 definition."""
import numpy as np
import pytest

from cache_util import device_step, make_step, run_plan
from gpu_util import require_gpu, to_np
from oracle import cache as oc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return require_gpu()


@pytest.fixture(scope="module")
def F(torch):
    from tree_forked_hybrid_gb300 import fork
    return fork


def inputs(torch, st, Hq, Hkv, d, seed, sharp=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    bf = lambda *s: torch.randn(s, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
    kc, vc = bf(st["n_pages"], Hkv, st["page"], d), bf(st["n_pages"], Hkv, st["page"], d)
    return bf(st["T_cap"], Hq, d) * sharp, kc, vc


def reference(torch, st, q, kc, vc, window, scale):
    """float64 on the GPU, one request at a time: (rows, sum of weight * |value|)."""
    q, kc, vc = q.double(), kc.double(), vc.double()
    Hq, Hkv, d = q.shape[1], kc.shape[1], q.shape[2]
    out, mag = torch.zeros_like(q), torch.zeros_like(q)
    row = 0
    for b, n in enumerate(np.maximum(st["n_new"], 0)):
        ln = int(st["length"][b])
        if n == 0:
            continue
        pages = torch.from_numpy(st["table"][b, :-(-(ln + n) // st["page"])].astype(np.int64)).cuda()
        K, V = (x[pages].transpose(0, 1).reshape(Hkv, -1, d)[:, :ln + n] for x in (kc, vc))
        see = torch.zeros((n, ln + n), dtype=torch.bool, device="cuda")
        paths = []
        for i in range(n):
            p = i - 1 if st["parent"] is None else int(st["parent"][row + i])
            paths.append((paths[p] if p >= 0 else []) + [i])
            t = ln + len(paths[i]) - 1
            see[i, (max(0, t - window + 1) if window else 0):ln] = True
            for depth, j in enumerate(paths[i]):
                see[i, ln + j] = not window or t - (ln + depth) < window
        see = see[:, None].expand(n, Hq // Hkv, -1).reshape(-1, ln + n)
        for g in range(Hkv):
            h = slice(g * (Hq // Hkv), (g + 1) * (Hq // Hkv))
            x = (q[row:row + n, h].reshape(-1, d) @ K[g].T) * scale
            x = x.masked_fill(~see, -torch.inf)
            w = torch.softmax(x, -1)
            # a masked value has no part in the sum, whatever it is
            out[row:row + n, h] = _weighted(torch, w, see, V[g]).reshape(n, -1, d)
            mag[row:row + n, h] = _weighted(torch, w, see, V[g].abs()).reshape(n, -1, d)
        row += n
    return out[:row], mag[:row]


def _weighted(torch, w, see, V):
    if bool(torch.isfinite(V).all()):
        return w @ V
    return torch.stack([(w[r][see[r]][:, None] * V[see[r]]).sum(0) for r in range(w.shape[0])])


def check(torch, got, want, mag):
    """bf16 weights (2^-8 of the sum of |weight * value| in the numerator, and as much by the denominator),
    float32 sums and an exponential of a few 2^-22 (below 2^-12 of that sum), one rounding of the result (2^-8 of it)."""
    tol = want.abs() * 2.0 ** -8 + mag * (2.0 ** -7 + 2.0 ** -12) + 1e-30
    err = (got.double() - want).abs()
    assert bool(torch.isfinite(got).all())
    assert bool((err <= tol).all()), float((err / tol).max())


def run(F, torch, st, q, kc, vc, Hq, Hkv, d, window=0, scale=None, max_new=None):
    c, a = device_step(torch, st, Hq, Hkv, d, max_new)
    run_plan(F, c, a)
    o = torch.full((st["T_cap"], Hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((F.fork_cache_attn_workspace_bytes(c),), 255, dtype=torch.uint8, device="cuda")  # NaN everywhere
    F.fork_cache_attn(c, q, kc, vc, o, window, scale, ws)
    assert F.fork_cache_status(c) == 0
    assert bool((o[st["T"]:] == 7).all())
    return o[:st["T"]], c


SHAPES = [  # Hq, Hkv, d, page
    (4, 1, 128, 16), (4, 4, 64, 32), (12, 4, 64, 64), (14, 2, 128, 128), (8, 1, 128, 256), (32, 1, 64, 16), (16, 2, 128, 64),
    (20, 4, 128, 32),
]
STEPS = [  # lengths, new tokens, tree
    ([1], [1], False), ([0], [1], True), ([127, 128, 129, 0, 383], [1, 1, 1, 1, 1], False),
    ([0, 700, 5, 64], [64, 1, 17, 33], True), ([250, 0, 90], [3, 0, 9], True), ([0, 300], [150, 40], False),
    ([1500, 40, 900, 3], [2, 4, 3, 1], True), ([126], [4], True), ([127], [64], True), ([0, 31], [129, 1], False),
]


@pytest.mark.parametrize("s", range(len(SHAPES)))
@pytest.mark.parametrize("k", range(len(STEPS)))
def test_matches_the_definition(F, torch, s, k):
    Hq, Hkv, d, page = SHAPES[s]
    length, n_new, tree = STEPS[k]
    st = make_step(10 * s + k, length, n_new, page, tree)
    q, kc, vc = inputs(torch, st, Hq, Hkv, d, s + k, sharp=1.0 + (k % 3))
    for window in (0, 1 + 40 * k, 3):
        got, _ = run(F, torch, st, q, kc, vc, Hq, Hkv, d, window, 0.1)
        check(torch, got, *reference(torch, st, q, kc, vc, window, 0.1))


def test_reference_against_the_oracle(F, torch):
    st = make_step(5, [40, 0], [7, 3], 16, True)
    q, kc, vc = inputs(torch, st, 4, 2, 64, 1)
    for W in (0, 5):
        want, _ = reference(torch, st, q, kc, vc, W, 0.2)
        n = lambda x: x.double().cpu().numpy()  # noqa: E731
        o = oc.attention(n(q), n(kc), n(vc), st["table"], st["length"], st["n_new"], st["parent"], 16, W, 0.2)
        np.testing.assert_allclose(n(want), o, atol=1e-12)


@pytest.mark.parametrize("Hq,Hkv,d,tree,n", [(4, 1, 128, True, 4), (16, 2, 64, False, 1), (8, 2, 128, True, 30)])
def test_long_contexts_are_split_and_joined(F, torch, Hq, Hkv, d, tree, n):
    """Few rows over many keys: every SM has a part of each row; an odd length; another request beside it."""
    st = make_step(9, [70001, 3, 20000], [n, 1, n], 64, tree)
    q, kc, vc = inputs(torch, st, Hq, Hkv, d, 3, sharp=2.0)
    got, _ = run(F, torch, st, q, kc, vc, Hq, Hkv, d)
    check(torch, got, *reference(torch, st, q, kc, vc, 0, d ** -0.5))


@pytest.mark.parametrize("R,n,tree", [(400, 1, False), (700, 3, True)])
def test_many_requests(F, torch, R, n, tree):
    """More items than threads of a CTA."""
    rng = np.random.default_rng(R)
    st = make_step(R, rng.integers(0, 300, R), np.where(rng.random(R) < 0.2, -1, n), 16, tree)
    st["length"][st["n_new"] < 0] = 0
    q, kc, vc = inputs(torch, st, 8, 2, 64, 3)
    got, _ = run(F, torch, st, q, kc, vc, 8, 2, 64)
    check(torch, got, *reference(torch, st, q, kc, vc, 0, 0.125))


def test_capacity_does_not_change_what_is_computed(F, torch):
    """The same step through the kernel forms for small and for large steps."""
    st = make_step(2, [200, 31], [2, 1], 16, True)
    q, kc, vc = inputs(torch, st, 4, 1, 128, 3)
    st["T_cap"], q = 80, torch.cat([q, q.new_zeros(80 - st["T_cap"], 4, 128)])
    st["parent"] = np.concatenate([st["parent"], np.full(80 - len(st["parent"]), -1, np.int32)])
    for max_new in (2, 4, 8, 16, 64, 80):
        got, _ = run(F, torch, st, q, kc, vc, 4, 1, 128, max_new=max_new)
        check(torch, got, *reference(torch, st, q, kc, vc, 0, 128 ** -0.5))


@pytest.mark.parametrize("max_new", [4, 8, 64])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), float("-inf")])
def test_odd_values_reach_only_the_rows_that_see_them(F, torch, max_new, d, what):
    """NaN and infinities behind the sequences' ends, in pages of no one, before a window, and in one drafted branch."""
    st = make_step(4, [200, 131, 60], [4, 3, 2], 16, True, T_cap=64)
    st["parent"][:4] = [-1, 0, 0, 2]
    st["parent"][4:7] = [-1, -1, 1]
    st["parent"][7:9] = [-1, -1]
    Hq, Hkv = 8, 2
    q, kc, vc = inputs(torch, st, Hq, Hkv, d, 3)
    clean_k, clean_v = kc.clone(), vc.clone()
    used = torch.zeros(st["n_pages"], 16, dtype=torch.bool, device="cuda")
    for b in range(3):
        for y in range(int(st["length"][b] + st["n_new"][b])):
            used[int(st["table"][b, y // 16]), y % 16] = True
    for x in (kc, vc):
        x.transpose(1, 2)[~used] = what
    got, _ = run(F, torch, st, q, kc, vc, Hq, Hkv, d, 0, None, max_new)
    check(torch, got, *reference(torch, st, q, clean_k, clean_v, 0, d ** -0.5))
    # a window: what lies before it is not seen by any row
    W = 50
    for b in range(3):
        for y in range(int(st["length"][b]) - W + 1):
            kc[int(st["table"][b, y // 16]), :, y % 16] = what
            vc[int(st["table"][b, y // 16]), :, y % 16] = what
    got, _ = run(F, torch, st, q, kc, vc, Hq, Hkv, d, W, None, max_new)
    check(torch, got, *reference(torch, st, q, clean_k, clean_v, W, d ** -0.5))
    # one branch's key and value: rows 1 (request 0) sees it, its siblings do not
    kc, vc = clean_k.clone(), clean_v.clone()
    y = 201
    page = int(st["table"][0, y // 16])
    vc[page, 0, y % 16, 5] = what
    kc[page, 1, y % 16, 7] = what
    got, _ = run(F, torch, st, q, kc, vc, Hq, Hkv, d, 0, None, max_new)
    want, mag = reference(torch, st, q, clean_k, clean_v, 0, d ** -0.5)
    hit = torch.zeros_like(got, dtype=torch.bool)
    hit[1, :Hq // Hkv, 5] = True
    hit[1, Hq // Hkv:] = True
    g = got.clone()
    g[hit] = want[hit].to(g.dtype)
    check(torch, g, want, mag)
    bad = got[1, :Hq // Hkv, 5]
    assert bool(torch.isnan(bad).all()) if what != what else bool((bad == what).all())


def test_chain_of_new_tokens_with_odd_values(F, torch):
    """A prompt chunk: an infinity in a later token's value does not reach earlier tokens."""
    st = make_step(4, [100], [40], 16, False)
    q, kc, vc = inputs(torch, st, 4, 1, 64, 3)
    clean = vc.clone()
    page = int(st["table"][0, 120 // 16])
    vc[page, 0, 120 % 16] = float("nan")
    got, _ = run(F, torch, st, q, kc, vc, 4, 1, 64)
    want, mag = reference(torch, st, q, kc, clean, 0, 0.125)
    check(torch, got[:20], want[:20], mag[:20])
    assert bool(torch.isnan(got[20:]).all())


def test_bits_do_not_depend_on_timing_or_the_batch_buffers(F, torch):
    st = make_step(8, [5000, 3000, 1], [5, 1, 2], 32, True)
    q, kc, vc = inputs(torch, st, 16, 4, 128, 1)
    first, _ = run(F, torch, st, q, kc, vc, 16, 4, 128)
    for _ in range(5):
        again, _ = run(F, torch, st, q, kc, vc, 16, 4, 128)
        assert torch.equal(first, again)


def test_in_place_stream_and_graph(F, torch):
    """o = q; a captured step (plan, append, attention) replayed for other lengths; two graphs of one workspace in turn."""
    Hq, Hkv, d, P, R = 8, 2, 64, 16, 3
    c = F.Cache(24, R, 8, 20, 64, P, Hq, Hkv, d)
    g = torch.Generator(device="cuda").manual_seed(0)
    rnd = lambda *s: torch.randn(s, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    perm = torch.randperm(64, generator=torch.Generator().manual_seed(1)).int().cuda()
    c.table.copy_(perm[:60].view(3, 20))
    length, n_new, blocks, ring, state = i32([100, 7, 300]), i32([1, 1, 1]), i32([20, 20, 20]), perm.clone(), i32([0, 0])
    bo, so = torch.empty_like(blocks), torch.empty_like(state)
    kc, vc = (rnd(64, Hkv, P, d) for _ in range(2))
    q, k, v = rnd(24, Hq, d), rnd(24, Hkv, d), rnd(24, Hkv, d)
    ws = torch.empty(F.fork_cache_attn_workspace_bytes(c), dtype=torch.uint8, device="cuda")
    rope = F.Rope(64)
    qr, o = torch.zeros_like(q), torch.zeros_like(q)

    def step(window):
        F.fork_cache_plan(c, length, n_new, None, blocks, bo, ring, state, so)
        F.fork_cache_append(c, rope, q, k, v, qr, kc, vc)
        F.fork_cache_attn(c, qr, kc, vc, o, window, None, ws)

    step(0)
    torch.cuda.synchronize()
    graphs = []
    for W in (0, 64):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            step(W)
        graphs.append((W, gr))
    for lens, new in (([100, 7, 300], [1, 1, 1]), ([0, 250, 31], [8, 0, 5]), ([19, 20, 21], [8, 8, 8])):
        length.copy_(i32(lens))
        n_new.copy_(i32(new))
        for W, gr in graphs:
            gr.replay()
            torch.cuda.synchronize()
            replayed = o.clone()
            o.zero_()
            step(W)
            assert F.fork_cache_status(c) == 0
            T = sum(new)
            assert torch.equal(replayed[:T], o[:T])
            st = dict(length=np.array(lens), n_new=np.array(new), parent=None, page=P, table=to_np(c.table))
            check(torch, o[:T], *reference(torch, st, qr, kc, vc, W, d ** -0.5))
    # in place, on a stream of its own
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    F.fork_cache_attn(c, qr, kc, vc, qr, 64, None, ws, stream=side)
    side.synchronize()
    assert torch.equal(qr[:T], o[:T])


def test_far_offsets(F, torch):
    """A pool whose last pages lie past 2^32 bytes and 2^31 elements."""
    P, Hkv, d, n_pages = 256, 2, 128, 33000  # 2.2e9 elements
    st = make_step(3, [600, 300], [2, 1], P, True)
    kc = torch.empty((n_pages, Hkv, P, d), dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    pages = torch.arange(n_pages - 6, n_pages, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(0)
    kc[pages] = torch.randn((6, Hkv, P, d), device="cuda", generator=g).to(torch.bfloat16)
    vc[pages] = torch.randn((6, Hkv, P, d), device="cuda", generator=g).to(torch.bfloat16)
    st["n_pages"], st["ring"] = n_pages, np.zeros(n_pages, np.int32)
    st["ring_in"] = np.array([0, 0], np.int32)
    st["table"] = np.array([[n_pages - 1, n_pages - 3, n_pages - 5], [n_pages - 2, n_pages - 6, -1]], np.int32)
    q = torch.randn((st["T_cap"], 8, d), device="cuda", generator=g).to(torch.bfloat16)
    got, c = run(F, torch, st, q, kc, vc, 8, Hkv, d)
    small = dict(st, table=st["table"] - (n_pages - 6) * (st["table"] >= 0))
    check(torch, got, *reference(torch, small, q, kc[pages], vc[pages], 0, d ** -0.5))
    k = torch.ones((st["T_cap"], Hkv, d), dtype=torch.bfloat16, device="cuda")
    F.fork_cache_append(c, None, None, k, k, None, kc, vc)
    assert int(to_np(c.tok_slot)[0]) // P == n_pages - 5
    assert float(kc[n_pages - 5, :, 600 - 512].float().sum()) == Hkv * d


def test_bad_page_and_argument_checks(F, torch):
    """A bad page reads as zeros; refusals."""
    st = make_step(1, [40], [1], 16, False)
    q, kc, vc = inputs(torch, st, 4, 1, 64, 0)
    st["table"][0, 1] = 10 ** 6
    c, a = device_step(torch, st, 4, 1, 64)
    run_plan(F, c, a)
    o = torch.zeros_like(q)
    F.fork_cache_attn(c, q, kc, vc, o)
    assert F.fork_cache_status(c) == F.FORK_STATUS_BAD_PAGE
    page = int(st["table"][0, 0])
    kc2, vc2 = torch.cat([kc, torch.zeros_like(kc[:1])]), torch.cat([vc, torch.zeros_like(vc[:1])])
    st["table"][0, 1] = kc.shape[0]
    want, mag = reference(torch, st, q, kc2, vc2, 0, 0.125)
    check(torch, o[:1], want, mag)
    assert page >= 0
    for bad in (dict(window=-1), dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf"))):
        with pytest.raises(F.ForkError):
            F.fork_cache_attn(c, q, kc, vc, o, **bad)
    with pytest.raises(F.ForkError):
        F.fork_cache_attn(c, q, kc, vc, o, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    for args in ((q.float(), kc, vc, o), (q, kc[:-1], vc, o), (q, kc, vc.transpose(0, 1), o), (q, kc, vc, o[1:])):
        with pytest.raises(ValueError):
            F.fork_cache_attn(c, *args)


@pytest.mark.parametrize("max_new", [1, 4, 64])
def test_a_wait_that_runs_out_is_reported_and_leaves_the_context_usable(F, torch, max_new):
    st = make_step(1, [3000, 40], [1, 1], 16, True, T_cap=64)
    q, kc, vc = inputs(torch, st, 8, 1, 128, 0)
    c, a = device_step(torch, st, 8, 1, 128, max_new)
    run_plan(F, c, a)
    clean = torch.zeros_like(q)
    F.fork_cache_attn(c, q, kc, vc, clean)
    assert F.fork_cache_status(c) == 0
    o = torch.zeros_like(q)
    c.set_wait_limit_us(2000)
    F.fork_cache_attn(c, q, kc, vc, o, flags=F.FORK_TEST_STALL)
    assert F.fork_cache_status(c) == F.FORK_STATUS_TIMEOUT
    c.set_wait_limit_us(0)
    run_plan(F, c, a)  # a plan clears the status
    F.fork_cache_attn(c, q, kc, vc, o)
    assert F.fork_cache_status(c) == 0
    assert torch.equal(o, clean)


@pytest.mark.parametrize("Hq,Hkv,d,page,length,n_new,tree", [
    (4, 1, 128, 16, [127, 128, 1, 383], [1, 1, 1, 1], False), (12, 4, 64, 64, [700, 5, 64], [3, 1, 5], True),
    (8, 8, 128, 32, [9000, 40], [1, 1], False), (32, 1, 64, 16, [2000, 31, 0], [1, 1, 1], False),
    (16, 2, 64, 32, [4001, 300], [4, 3], True), (7, 1, 128, 128, [600, 3], [2, 1], True)])
def test_few_rows_carry_their_weights_in_more_than_bf16(F, torch, Hq, Hkv, d, page, length, n_new, tree):
    """The kernel for few rows: a weight is the largest bf16 number below it and the bf16 of the rest, which is off by 2^-8
    of at most 2^-7 of it; sums, scores and exponential within 2^-12 as in `check`; one rounding of the result."""
    st = make_step(31, length, n_new, page, tree)
    for sharp in (1.0, 3.0):
        q, kc, vc = inputs(torch, st, Hq, Hkv, d, 5, sharp)
        for window in (0, 100):
            got, _ = run(F, torch, st, q, kc, vc, Hq, Hkv, d, window)
            want, mag = reference(torch, st, q, kc, vc, window, d ** -0.5)
            tol = want.abs() * 2.0 ** -8 + mag * (2.0 ** -15 + 2.0 ** -12) + 1e-30
            err = (got.double() - want).abs()
            assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("max_new", [1, 8, 64])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("what", [float("inf"), float("-inf")])
def test_an_infinity_that_every_row_sees(F, torch, max_new, d, what):
    """In a tile without masked keys: the sum is that infinity, whatever the weight (1 where the queries are zero)."""
    st = make_step(4, [1000, 300], [1, 1], 16, False, T_cap=64)
    q, kc, vc = inputs(torch, st, 8, 2, d, 3)
    for b, y in ((0, 5), (0, 700), (1, 130)):
        vc[int(st["table"][b, y // 16]), :, y % 16, 3 + b] = what
    for qq in (q, torch.zeros_like(q)):
        got, _ = run(F, torch, st, qq, kc, vc, 8, 2, d, 0, None, max_new)
        for b in range(2):
            assert bool((got[b, :, 3 + b] == what).all())
            assert bool(torch.isfinite(got[b, :, :3 + b]).all()) and bool(torch.isfinite(got[b, :, 4 + b:]).all())


@pytest.mark.parametrize("Hq,Hkv,d,n,tree", [(4, 1, 128, 2, False), (16, 2, 64, 4, True), (16, 2, 128, 9, True), (8, 1, 64, 40, False)])
def test_the_last_positions(F, torch, Hq, Hkv, d, n, tree):
    """A windowed layer far along a stream, up to the last cache index that the handle allows (2^31 - 65): the bits of the
    same step 2^31 - 2048 tokens earlier (pages before the window are not read)."""
    P, far, W = 64, 2 ** 31 - 2048, 300
    for end in (2048 - 64, 2048 - 64 - 70, 2048 - 128):  # the last tile half full, of one key or so, full
        st = make_step(6, [end - n], [n], P, tree, n_pages=40)
        q, kc, vc = inputs(torch, st, Hq, Hkv, d, 2)
        want, _ = run(F, torch, st, q, kc, vc, Hq, Hkv, d, W)
        check(torch, want, *reference(torch, st, q, kc, vc, W, d ** -0.5))
        _, a = device_step(torch, st, Hq, Hkv, d)
        c = F.Cache(st["T_cap"], 1, st["max_new"], (2 ** 31 - 1) // P, st["n_pages"], P, Hq, Hkv, d)
        c.table[0, far // P:far // P + st["table"].shape[1]] = torch.from_numpy(st["table"][0]).cuda()
        a["length"] += far
        a["blocks_in"] += far // P
        run_plan(F, c, a)
        o = torch.zeros_like(q)
        F.fork_cache_attn(c, q, kc, vc, o, W)
        assert F.fork_cache_status(c) == 0
        assert torch.equal(o[:n], want), end
