"""Serving steps over the paged cache as they are used: plan, append, attention, sampling, keep."""
import math

import numpy as np
import pytest

from gpu_util import require_gpu, to_np
from oracle import cache as oc
from test_gpu_cache_attn import check, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return require_gpu()


@pytest.fixture(scope="module")
def F(torch):
    from tree_forked_hybrid_gb300 import fork
    return fork


@pytest.mark.parametrize("tree,max_new,page", [(True, 12, 16), (False, 30, 32), (True, 4, 64)])
def test_steps_grow_shrink_and_finish(F, torch, tree, max_new, page):
    """Random requests over steps; the cache always holds the kept tokens' keys at their positions, and every attention
    row equals the definition on what the cache holds."""
    from tree_forked_hybrid_gb300 import workloads as wl
    from tree_forked_hybrid_gb300.runner import CacheRound
    shapes = (wl.AttnShape("full", 8, 2, 64, 0, 1e4), wl.AttnShape("window", 8, 2, 64, 20, 5e5))
    R, V = 5, 997
    cr = CacheRound(shapes, T_cap=R * max_new, max_req=R, max_new=max_new, max_blocks=200 // page + 1, n_pages=R * (200 // page + 1),
                    page_tokens=page)
    rng = np.random.default_rng(max_new)
    g = torch.Generator(device="cuda").manual_seed(1)
    emb = {a.name: [torch.randn((V, h, 64), device="cuda", generator=g).to(torch.bfloat16) for h in (8, 2, 2)] for a in shapes}
    head = torch.randn((8 * 64, V), device="cuda", generator=g)
    held = [[] for _ in range(R)]  # the kept tokens of every request
    for step in range(12):
        n_new = rng.integers(0, max_new + 1, R)
        n_new[rng.random(R) < 0.15] = -1
        n_new[[len(h) + max_new > 190 for h in held]] = -1
        n = np.maximum(n_new, 0)
        tokens = rng.integers(0, V, (int(n.sum()),))
        parent, r = np.full(R * max_new, -1, np.int32), 0
        for k in n:
            for i in range(k):
                parent[r + i] = rng.integers(max(-1, i - 4), i) if tree else i - 1
            r += k
        T = r
        cr.plan(torch.from_numpy(n_new.astype(np.int32)), torch.from_numpy(parent) if tree else None)
        ids = torch.from_numpy(tokens).cuda()
        for a in shapes:
            for name, e in zip("qkv", emb[a.name]):
                cr.inputs[a.name][name][:T] = e[ids]
        cr.run()
        assert cr.status() == 0
        st = dict(length=np.array([len(h) for h in held]), n_new=n_new, parent=parent if tree else None, page=page,
                  table=to_np(cr.cache.table))
        for a in shapes:
            f, amp = oc.rope_freq(64, a.rope_theta)
            q = oc.rope(to_np(cr.inputs[a.name]["q"])[:T], to_np(cr.cache.tok_pos)[:T], 64, False, f, amp)
            q = torch.from_numpy(q).cuda().to(torch.bfloat16)
            kc, vc = cr.kv[a.name]
            # (the buffer of rotated queries holds the last layer's: the reference takes the kernel's own, which may round
            # a value next to a border the other way)
            if a is shapes[-1]:
                q_rot = cr.q_rot[:T]
                assert bool(((q_rot.float() - q.float()).abs() <= q.float().abs() * 2.0 ** -7 + 1e-5).all())
                check(torch, cr.attn_out[a.name][:T], *reference(torch, st, q_rot, kc, vc, a.window, 0.125))
            # the kept tokens' keys and values, wherever their pages are
            for b in range(R):
                if n_new[b] < 0 or not held[b]:
                    continue
                y = np.arange(len(held[b]))
                pages, off = st["table"][b, y // page], y % page
                want = oc.rope(to_np(emb[a.name][1][held[b]]), y, 64, False, f, amp)
                got = to_np(kc[pages, :, off])
                assert (np.abs(got - want) <= np.abs(want) * 2.0 ** -8 + 1e-5 * 8).all()
                assert torch.equal(vc[pages, :, off], emb[a.name][2][held[b]])
        # a token drawn at every row
        logits = cr.attn_out["full"][:T].reshape(T, -1).float() @ head
        u = torch.rand(T, device="cuda", generator=g)
        par = dict(top_k=torch.full((T,), 50, dtype=torch.int32, device="cuda"), temperature=torch.full((T,), 2.0, device="cuda"))
        drawn = cr.sample(logits, u, **par).tolist()
        assert drawn == [oc.sample_row(logits[t].cpu().numpy(), float(u[t]), 2.0, 50)[0] for t in range(T)]
        # what is kept: a path of the tree, or the first tokens
        n_keep, paths, r = [], [], 0
        for b in range(R):
            if n_new[b] < 0:
                held[b] = []
            path = []
            if n[b]:
                j = int(rng.integers(n[b]))
                while j >= 0:
                    path.insert(0, j)
                    j = int(parent[r + j])
            n_keep.append(len(path))
            paths.append(path)
            held[b] = held[b] + [int(tokens[r + j]) for j in path]
            r += n[b]
        cr.keep(n_keep, paths if tree else None)
        assert cr.length.tolist() == [len(h) for h in held]


def test_a_chunk_equals_the_round(F, torch):
    """A trunk cached in chunks, then questions as chains: the rows of fork_attn on the same stream."""
    from tree_forked_hybrid_gb300 import workloads as wl
    from tree_forked_hybrid_gb300.runner import CacheRound, DeviceRound
    rnd = wl.make_round(1)
    dr = DeviceRound(rnd)
    dr.run()
    a = rnd.attn_shapes[0]
    P0 = int(rnd.trunk_len[0])
    nq, ql = int(rnd.n_q[0]), [int(x) for x in rnd.q_len[:int(rnd.n_q[0])]]
    inp = dr.inputs[a.name]
    first_q = int(rnd.trunk_len.sum())
    cr = CacheRound((a,), T_cap=256, max_req=1, max_new=256, max_blocks=16, n_pages=16, page_tokens=64)

    def feed(lo, n):
        cr.plan(torch.tensor([n], dtype=torch.int32))
        for k in "qkv":
            cr.inputs[a.name][k][:n] = inp[k][lo:lo + n]
        cr.run()
        assert cr.status() == 0
        d = (cr.attn_out[a.name][:n].float() - dr.attn_out[a.name][lo:lo + n].float()).abs().max()
        assert float(d) <= 2e-2  # both kernels' tolerance against the definition, unit-variance inputs
    at = 0
    for n in (100, 256, 1, P0):
        n = min(n, P0 - at)
        if n > 0:
            feed(at, n)
            cr.keep([n])
            at += n
    assert at == P0
    for i in range(nq):  # every question from the trunk's end: nothing of the last one is kept
        feed(first_q + sum(ql[:i]), ql[i])


def small_round(torch):
    from tree_forked_hybrid_gb300 import workloads as wl
    from tree_forked_hybrid_gb300.runner import CacheRound
    cr = CacheRound((wl.AttnShape("full", 4, 2, 64, 0, 1e4),), T_cap=24, max_req=2, max_new=12, max_blocks=3, n_pages=4, page_tokens=16)
    g = torch.Generator(device="cuda").manual_seed(3)
    for x in cr.inputs["full"].values():
        x.copy_(torch.randn(x.shape, device="cuda", generator=g))
    return cr


def test_keep_refuses(F, torch):
    """Nothing is moved or kept after a failed step, or for tokens that the step did not have."""
    cr = small_round(torch)
    tree = torch.tensor([-1, 0, 0, -1] + [-1] * 20, dtype=torch.int32)
    cr.plan(torch.tensor([3, 1], dtype=torch.int32), tree)
    cr.run()
    before = [x.clone() for x in cr.kv["full"]]
    for n_keep, path in (([4, 0], None), ([-1, 0], None), ([1], None), ([2, 0], [[0], []]), ([2, 0], [[0, 3], []]),
                         ([2, 0], [[-1, 0], []])):
        with pytest.raises(ValueError):
            cr.keep(n_keep, path)
    assert cr.length.tolist() == [0, 0]
    cr.keep([2, 1], [[0, 2], [0]])
    assert cr.length.tolist() == [2, 1]
    before = [x.clone() for x in cr.kv["full"]]
    cr.plan(torch.tensor([13, 0], dtype=torch.int32))  # above max_new: refused
    cr.run()
    with pytest.raises(RuntimeError, match="BAD_DESC"):
        cr.keep([2, 0], [[0, 2], []])
    assert cr.length.tolist() == [2, 1]
    assert all(torch.equal(x, y) for x, y in zip(cr.kv["full"], before))


def test_steps_on_another_stream(F, torch):
    """plan, run and sample on a stream of their own, behind work that is queued there: the same bits."""
    out = []
    for other in (False, True):
        cr = small_round(torch)
        s = torch.cuda.Stream() if other else None
        n_new, tree = torch.tensor([5, 9], dtype=torch.int32).cuda(), torch.tensor([-1, 0, 0, 1, -1, -1, 0, 1, 1, 3, 4, 4, 0, 7] + [-1] * 10, dtype=torch.int32).cuda()
        u, t = torch.linspace(0.05, 0.95, 14, device="cuda"), torch.full((14,), 0.7, device="cuda")
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            x = torch.ones((2048, 2048), device="cuda")
            for _ in range(8):
                x = x @ x * 1e-4  # (keeps the stream busy for a while)
        cr.plan(n_new, tree, stream=s)
        cr.run(stream=s)
        with torch.cuda.stream(s):
            logits = cr.attn_out["full"][:14].reshape(14, -1).float()
        token = cr.sample(logits, u, stream=s, temperature=t)
        torch.cuda.synchronize()
        out.append((cr.attn_out["full"].clone(), token.clone(), cr.kv["full"][0].clone()))
    assert all(torch.equal(a, b) for a, b in zip(*out))


@pytest.mark.parametrize("T_cap", [40, 2100])  # the plan in one launch and in two
@pytest.mark.parametrize("fault", ["parent", "page"])
@pytest.mark.parametrize("call", ["keep", "status", "nothing"])
def test_a_request_ends_in_a_step_that_fails(F, torch, T_cap, fault, call):
    """The plan returned its pages before the step failed: its slot takes a new prompt, whatever is called in between."""
    from tree_forked_hybrid_gb300 import workloads as wl
    from tree_forked_hybrid_gb300.runner import CacheRound
    cr = CacheRound((wl.AttnShape("full", 4, 2, 64, 0, 1e4),), T_cap=T_cap, max_req=3, max_new=20, max_blocks=4, n_pages=9, page_tokens=16)
    g = torch.Generator(device="cuda").manual_seed(3)
    for x in cr.inputs["full"].values():
        x.copy_(torch.randn(x.shape, device="cuda", generator=g))
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    cr.plan(i32(20, 10, 3))
    cr.run()
    cr.keep([20, 10, 3])
    parent = torch.full((T_cap,), -1, dtype=torch.int32)
    state = [x.clone() for x in (*cr.kv["full"], cr.q_rot, cr.attn_out["full"])]
    page = int(cr.cache.table[1, 0])
    if fault == "parent":
        parent[2] = 5
    else:
        cr.cache.table[1, 0] = 10 ** 6
    cr.plan(i32(-1, 4, 0), parent)
    cr.run()
    if fault == "parent":  # what follows a refused tree does nothing
        assert all(torch.equal(x, y) for x, y in zip(state, (*cr.kv["full"], cr.q_rot, cr.attn_out["full"])))
    if call == "keep":
        with pytest.raises(RuntimeError, match="BAD_DESC" if fault == "parent" else "BAD_PAGE"):
            cr.keep([0, 1, 0], [[], [0], []])
        assert cr.length.tolist() == [0, 10, 3]
    elif call == "status":
        assert cr.status() == (0x1 if fault == "parent" else F.FORK_STATUS_BAD_PAGE)
    assert cr.blocks.tolist() == [0, 1, 1]
    cr.cache.table[1, 0] = page
    cr.plan(i32(18, 2, 1))
    cr.run()
    assert cr.status() == 0
    assert to_np(cr.cache.kv_len).tolist() == [18, 12, 4] and to_np(cr.cache.tok_pos)[:21].tolist() == [*range(18), 10, 11, 3]
    cr.keep([18, 2, 1])
    assert cr.length.tolist() == [18, 12, 4]


def test_a_request_ends_in_a_refused_step(F, torch):
    """Refused as a whole: nothing went back, the length stays."""
    cr = small_round(torch)
    cr.plan(torch.tensor([3, 1], dtype=torch.int32))
    cr.run()
    cr.keep([3, 1])
    cr.plan(torch.tensor([-1, 13], dtype=torch.int32))  # above max_new
    with pytest.raises(RuntimeError, match="BAD_DESC"):
        cr.keep([0, 0])
    assert cr.length.tolist() == [3, 1] and cr.blocks.tolist() == [1, 1]
    cr.plan(torch.tensor([1, 1], dtype=torch.int32))
    cr.run()
    cr.keep([1, 1])
    assert cr.length.tolist() == [4, 2]


def test_keep_refuses_what_is_no_path(F, torch):
    """Kept tokens have their keys rotated for the places that they are moved to only if they follow one another."""
    cr = small_round(torch)
    tree = torch.tensor([-1, 0, 0, 1, 3, -1, -1] + [-1] * 17, dtype=torch.int32)  # 0 -> (1 -> 3 -> 4, 2), 5; and a single one
    cr.plan(torch.tensor([6, 1], dtype=torch.int32), tree)
    cr.run()
    for path in ([1, 0], [0, 0], [0, 1, 1], [1], [0, 3], [1, 3], [0, 2, 3], [0, 5], [0, 1, 2], [2, 0, 1]):
        with pytest.raises(ValueError):
            cr.keep([len(path), 0], [path, []])
    for n in (3, 4):  # 0, 1, 2: the first tokens are not a path either
        with pytest.raises(ValueError):
            cr.keep([n, 0])
    assert cr.length.tolist() == [0, 0]
    k0, slot = cr.kv["full"][0].clone(), to_np(cr.cache.tok_slot)
    cr.keep([4, 1], [(0, 1, 3, 4), np.array([0])])
    assert cr.length.tolist() == [4, 1]
    for to, was in enumerate((0, 1, 3, 4)):
        a, b = divmod(int(slot[to]), 16), divmod(int(slot[was]), 16)
        assert torch.equal(cr.kv["full"][0][a[0], :, a[1]], k0[b[0], :, b[1]])
    # a chain after a tree: its first tokens alone (the parents of the step before do not count)
    cr.plan(torch.tensor([4, 0], dtype=torch.int32))
    cr.run()
    for path in ([1], [0, 2], [1, 0], [0, 0]):
        with pytest.raises(ValueError):
            cr.keep([len(path), 0], [path, []])
    cr.keep([3, 0], [[0, 1, 2, 3], []])
    assert cr.length.tolist() == [7, 1]
    # the first tokens of a tree that is a chain; 64 of them, the mask's last bit
    from tree_forked_hybrid_gb300 import workloads as wl
    from tree_forked_hybrid_gb300.runner import CacheRound
    cr = CacheRound((wl.AttnShape("full", 4, 2, 64, 0, 1e4),), T_cap=70, max_req=1, max_new=64, max_blocks=8, n_pages=8, page_tokens=16)
    cr.plan(torch.tensor([64], dtype=torch.int32), torch.arange(-1, 69, dtype=torch.int32))
    cr.keep([64])
    assert cr.length.tolist() == [64]


def test_a_step_is_kept_once(F, torch):
    cr = small_round(torch)
    cr.plan(torch.tensor([3, 2], dtype=torch.int32))
    cr.run()
    cr.keep([2, 1])
    for n_keep in ([1, 0], [2, 1], [0, 1]):
        with pytest.raises(ValueError):
            cr.keep(n_keep)
    cr.keep([0, 0])
    assert cr.length.tolist() == [2, 1]
    # captured with the rest of a step: every replay is a step of its own
    n_new = torch.tensor([1, 2], dtype=torch.int32).cuda()
    cr.plan(n_new)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        cr.plan(n_new)
        cr.run()
    for k in range(3):
        gr.replay()
        cr.keep([1, 2])
        assert cr.length.tolist() == [3 + k, 3 + 2 * k]


def test_plan_refuses_other_shapes(F, torch):
    """One count for every request and one parent for every row; nothing is spread or cut silently."""
    cr = small_round(torch)
    cr.plan(torch.tensor([3, 1], dtype=torch.int32))
    cr.run()
    cr.keep([3, 1])
    for n_new, parent in ((torch.tensor([1]), None), (torch.tensor(1), None), (torch.tensor([[1, 1]]), None), (torch.tensor([1.5, 1.0]), None),
                          (torch.tensor([1, 1, 1]), None), (torch.tensor([1, 1]), torch.tensor([-1])),
                          (torch.tensor([1, 1]), torch.full((25,), -1)), (torch.tensor([1, 1]), torch.full((24,), -1.0))):
        with pytest.raises(ValueError):
            cr.plan(n_new, parent)
    assert cr.n_new.tolist() == [3, 1] and cr.length.tolist() == [3, 1]
    cr.plan(torch.tensor([2, 1]), torch.tensor([-1, 0] + [-1] * 22))  # (64-bit counts and parents do)
    cr.run()
    cr.keep([2, 1])
    assert cr.length.tolist() == [5, 2]


def test_the_rounds_own_counts_are_planned_again(F, torch):
    """n_new filled once, a captured plan of it replayed: a token for every request in every step."""
    cr = small_round(torch)
    cr.n_new.fill_(1)
    cr.plan(cr.n_new)
    cr.run()
    cr.keep([1, 1])
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        cr.plan(cr.n_new)
        cr.run()
    for k in range(4):
        gr.replay()
        cr.keep([1, 1])
        assert cr.length.tolist() == [2 + k, 2 + k] and cr.n_new.tolist() == [1, 1]
