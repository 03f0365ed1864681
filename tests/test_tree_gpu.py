"""Attention of drafted trees over the ring cache, commit and advance, against the
definition in 64 bits and against ordinary decode steps."""
import numpy as np
import pytest
import torch

import tree_reference as ref
from helpers import f64, tol_for

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _rswa():
    from ring_sliding_window_b200 import rswa
    return rswa


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Case:
    def __init__(self, dtype, d, H, W, plens, t, T, n=None, parents=None, seed=1, layers=1,
                 scale=0.0, tail=None):
        rswa = _rswa()
        self.B, self.T, self.H, self.d, self.W = len(plens), T, H, d, W
        self.model = ref.Model(plens, W, H, d, dtype, seed).generate(t)
        self.st = rswa.State(self.B, layers, H, d, W, plens, dtype=dtype, n_generated=t,
                             scale=scale)
        for layer in range(layers):
            self.model.fill(self.st, layer)
        rng = np.random.default_rng(seed)
        self.n = [T] * self.B if n is None else list(n)
        self.parents = [ref.random_parents(rng, T) for _ in plens] if parents is None else parents
        self.q, self.k, self.v = (self.model.draw(self.B, T, H, d) for _ in range(3))
        self.scale = scale or d ** -0.5
        self.tree = self.st.tree(T)

    def run(self, layer=0):
        out = torch.full((self.B, self.T, self.H, self.d), 7.0, dtype=self.model.dtype,
                         device="cuda")
        self.tree.set(_ints(self.parents), _ints(self.n))
        self.tree.attention(layer, self.q.cuda(), self.k.cuda(), self.v.cuda(), out)
        torch.cuda.synchronize()
        assert self.st.check() == 0
        return out.cpu()

    def check(self, out, swa=False, rows=None):
        m = self.model
        for b in range(self.B):
            for i in range(self.T):
                if i >= self.n[b]:
                    assert bool((out[b, i] == 7.0).all()), "a row that holds no draft was written"
                    continue
                if rows is not None and i not in rows:
                    continue
                path = ref.path_of(self.parents[b], i)
                for h in range(self.H):
                    k, v = m.entries(b, h, [self.k[b, x] for x in path],
                                     [self.v[b, x] for x in path], swa)
                    o, mass = ref.attend(self.q[b, i, h], k, v, self.scale)
                    err = (out[b, i, h].double() - o).abs()
                    lim = ref.tolerance(o, mass, m.dtype)
                    assert bool((err <= lim).all()), (b, i, h, float((err / lim).max()))


KINDS = [(BF, 128), (BF, 64), (F32, 128), (F32, 64)]


@pytest.mark.parametrize("dtype,d", KINDS)
@pytest.mark.parametrize("T,W,plens,t", [
    (1, 8, (5,), (0,)),                    # one draft, nothing generated yet
    (1, 128, (1088,), (500,)),
    (4, 1, (3, 0), (2, 1)),                # the window holds the draft alone
    (8, 8, (0, 1, 130), (3, 8, 9)),        # no prompt; rings part full, full, wrapped
    (17, 5, (100, 64), (4, 23)),           # paths deeper than the window
    (33, 128, (257, 63, 128), (127, 128, 300)),
    (64, 100, (200,), (37,)),
    (65, 40, (190, 7), (55, 41)),
    (128, 129, (255,), (260,)),
    (128, 16, (65,), (10,)),
])
def test_tree_matches_the_definition(dtype, d, T, W, plens, t):
    rng = np.random.default_rng(T)
    n = [T] + [int(rng.integers(0, T + 1)) for _ in plens[1:]]
    c = Case(dtype, d, 2, W, plens, t, T, n=n)
    c.check(c.run())


@pytest.mark.parametrize("dtype,d", KINDS)
@pytest.mark.parametrize("parents", ["chain", "star", "pairs"])
def test_tree_shapes(dtype, d, parents):
    T = 40
    p = {"chain": [i - 1 for i in range(T)], "star": [-1] * T,
         "pairs": [(i - 1) // 2 if i else -1 for i in range(T)]}[parents]
    c = Case(dtype, d, 3, 24, (150, 31), (30, 5), T, parents=[p, p])
    c.check(c.run())


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
def test_tree_over_many_tiles_and_pieces(dtype, d):
    """Long prompts: rings split over several CTAs, CTAs holding parts of several rings."""
    c = Case(dtype, d, 2, 128, (5000, 17, 1300), (700, 3, 128), 24, n=(24, 9, 0))
    c.check(c.run(), rows=(0, 3, 8, 23))


@pytest.mark.parametrize("T", [7, 64, 128])
def test_tree_at_serving_sizes(T):
    """Every SM at work on long prompts, the caches in HBM, again and again: no wait runs out,
    and every pass gives the same."""
    rswa = _rswa()
    B, H, d, P, L = 4, 10, 128, 16000, 6
    st = rswa.State(B, L, H, d, 128, [P] * B, dtype=BF, n_generated=[1000] * B)
    g = torch.Generator(device="cuda").manual_seed(T)
    for x in st.k_cache + st.v_cache:
        x.normal_(generator=g)
    q, k, v = (torch.randn(B, T, H, d, generator=g, device="cuda").to(BF) for _ in range(3))
    tree = st.tree(T)
    first = [None] * L
    for _ in range(5):
        tree.set()
        for layer in range(L):
            out = torch.empty_like(q)
            tree.attention(layer, q, k, v, out)
            if first[layer] is None:
                first[layer] = out
            assert torch.equal(first[layer], out)
    assert st.check() == 0
    # the first draft of a chain, over the prompt, all but one of the ring, and itself
    for layer in (0, L - 1):
        for b, h in ((0, 0), (B - 1, H - 1)):
            keep = [s for s in range(P + 128) if s != P + 1000 % 128]
            ks, vs = (torch.cat([st.cache_view(layer, w, b, h)[keep], x[b, :1, h]]).double()
                      for w, x in (("k", k), ("v", v)))
            o, mass = ref.attend(q[b, 0, h], ks, vs, d ** -0.5)
            err = (first[layer][b, 0, h].double() - o).abs()
            assert bool((err <= ref.tolerance(o, mass, BF)).all())


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F32, 64)])
def test_tree_with_more_rings_than_ctas(dtype, d):
    B = 90
    plens = tuple(int(x) for x in np.random.default_rng(3).integers(0, 300, B))
    t = tuple(int(x) for x in np.random.default_rng(4).integers(0, 40, B))
    n = [int(x) for x in np.random.default_rng(5).integers(0, 12, B)]
    c = Case(dtype, d, 4, 16, plens, t, 11, n=n)
    c.check(c.run(), rows=(0, 5, 10))


@pytest.mark.parametrize("dtype,d", KINDS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_values_a_draft_does_not_see_never_reach_it(dtype, d, bad):
    """Non-finite keys and values in a sibling branch, in a ring entry that deeper drafts have
    outlived, and in rows behind the last draft: only the drafts that see them change."""
    T, W, P = 12, 10, 140
    parents = [[-1, 0, 1, 2, -1, 4, 5, 6, 7, 8, 9, 10]]
    c = Case(dtype, d, 2, W, (P,), (25,), T, n=(T - 1,), parents=parents, seed=5)
    clean = c.run()
    c.check(clean)
    # draft 4 and its branch (4..10) hold the bad value; drafts 0..3 do not see it
    c.k[0, 4, :, 3] = bad
    c.v[0, 4, :, 5] = bad
    c.v[0, T - 1] = bad
    c.k[0, T - 1] = bad
    out = c.run()
    assert torch.equal(out[:, :4], clean[:, :4])
    assert not bool(torch.isfinite(out[0, 5, :, 5]).any())
    # token 15 (slot P + 25 mod 10, which token 25 would overwrite): seen by no draft
    c = Case(dtype, d, 2, W, (P,), (25,), T, parents=parents, seed=6)
    clean = c.run()
    for h in range(2):
        c.st.cache_view(0, "v", 0, h)[P + 5, 7] = bad
        c.st.cache_view(0, "k", 0, h)[P + 5, 9] = bad
    assert torch.equal(c.run(), clean)
    # token 16, the oldest that a draft at depth 0 (token 25) sees; deeper ones do not
    for h in range(2):
        c.st.cache_view(0, "v", 0, h)[P + 6, 7] = bad
    out = c.run()
    shallow = [0, 4]
    deep = [i for i in range(T) if i not in shallow]
    assert torch.equal(out[:, deep], clean[:, deep])
    # the drafts that see it: that element alone takes the value on
    assert not bool(torch.isfinite(out[0, shallow, :, 7]).any())
    others = [e for e in range(d) if e != 7]
    assert torch.equal(out[:, shallow][..., others], clean[:, shallow][..., others])


@pytest.mark.parametrize("dtype,d", KINDS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_values_that_every_draft_sees_reach_it(dtype, d, bad):
    """A non-finite value in the prompt: that element takes it on, the others keep theirs."""
    c = Case(dtype, d, 2, 16, (700,), (5,), 9, seed=7)
    clean = c.run()
    for h in range(2):
        c.st.cache_view(0, "v", 0, h)[130, 7] = bad
    out = c.run()
    assert torch.equal(out[..., 7], torch.full_like(out[..., 7], bad)) or \
        (bad != bad and bool(out[..., 7].isnan().all()))
    others = [e for e in range(d) if e != 7]
    assert torch.equal(out[..., others], clean[..., others])


@pytest.mark.parametrize("dtype,d,T", [(BF, 128, 4), (BF, 64, 20), (BF, 128, 40), (BF, 64, 100),
                                       (F32, 128, 4), (F32, 64, 20)])
def test_dropped_copies_end_with_a_timeout_status(dtype, d, T):
    """With the kernel's cache copies dropped every wait runs out, and says so."""
    rswa = _rswa()
    c = Case(dtype, d, 1, 8, (200, 30), (3, 9), T)
    c.run()
    q, k, v = c.q.cuda(), c.k.cuda(), c.v.cuda()
    out = torch.empty_like(q)
    rswa.rswa_debug_inject_fault(c.st.handle, rswa.RSWA_FAULT_DROP_DECODE_COPIES)
    c.tree.attention(0, q, k, v, out)
    assert c.st.check() == rswa.RSWA_ETIMEOUT
    rswa.rswa_debug_inject_fault(c.st.handle, 0)
    c.check(c.run())


@pytest.mark.parametrize("dtype,d", KINDS)
def test_large_scores(dtype, d):
    """Scores of hundreds, growing along the keys: the running maximum moves at every tile."""
    c = Case(dtype, d, 2, 16, (700,), (20,), 9, seed=8)
    m = c.model
    ramp = torch.linspace(0, 40, 700)[:, None, None]
    m.pk[0] = (m.pk[0].float() * 0.05 + ramp * torch.sign(c.q[0, 0].float()) / d ** 0.5).to(dtype)
    m.fill(c.st)
    c.check(c.run())


@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("T,plens,t", [(3, (40, 300), (2, 50)), (16, (2000,), (9,)),
                                       (20, (500, 129), (0, 70)), (64, (700, 30), (20, 33)),
                                       (100, (900,), (64,)), (7, (9000,), (100,))])
@pytest.mark.parametrize("growing", [False, True])
def test_both_halves_of_a_weight_count(d, T, plens, t, growing):
    """bf16 against the bound that weights as pairs keep and single bf16 weights do not
    (test_tree_evict_cpu.py): values of one sign, so nothing cancels, rings in one piece and in
    several, and scores that grow along the keys, where the subtracted maximum moves and both
    halves of the sums so far are scaled."""
    c = Case(BF, d, 2, 64, plens, t, T, seed=40 + T)
    m = c.model
    for b, P in enumerate(plens):
        m.pv[b] = m.pv[b].abs()
        m.gv[b] = [x.abs() for x in m.gv[b]]
        if growing:
            ramp = torch.linspace(0, 60, P)[:, None, None]
            m.pk[b] = (m.pk[b].float() * 0.05 +
                       ramp * torch.sign(c.q[b, 0].float()) / d ** 0.5).to(BF)
    c.v = c.v.abs()
    m.fill(c.st)
    out = c.run()
    for b in range(len(plens)):
        for i in sorted({0, 1, T // 2, T - 1}):
            path = ref.path_of(c.parents[b], i)
            for h in range(2):
                k, v = m.entries(b, h, [c.k[b, x] for x in path], [c.v[b, x] for x in path])
                o, mass = ref.attend(c.q[b, i, h], k, v, c.scale)
                err = (out[b, i, h].double() - o).abs()
                lim = ref.pair_tolerance(c.q[b, i, h], k, o, mass, c.scale)
                assert bool((err <= lim).all()), (b, i, h, float((err / lim).max()))


@pytest.mark.parametrize("dtype,d", KINDS)
@pytest.mark.parametrize("rope", [0, 1, 2])
@pytest.mark.parametrize("swa", [False, True])
def test_chain_verify_and_commit_equals_decode_steps(dtype, d, rope, swa):
    """A chain of drafts gives what as many decode steps give, layer by layer, and after the
    commit the caches, counters and next step are the same: across ring wraps."""
    rswa = _rswa()
    B, L, H, W, plens, T = 2, 2, 3, 12, (150, 20), 9
    a, b = (rswa.State(B, L, H, d, W, plens, dtype=dtype) for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(3)

    def draw(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)

    for st in (a, b):
        if rope:
            st.set_rope(rope)
        if swa:
            st.set_attention(rswa.RSWA_ATTN_STANDARD_SWA)
    tot = sum(plens)
    for layer in range(L):
        q, k, v = (draw(tot, H, d) for _ in range(3))
        for st in (a, b):
            st.prefill(layer, q, k, v, torch.empty_like(q))
    tree = b.tree(T)
    # two roundings of a weight and of the output on either side; rope rounds q on the tree's
    tol = (2e-2 if dtype == BF else 1e-5)
    for step in range(4):
        qs, ks, vs = ([draw(B, T, H, d) for _ in range(L)] for _ in range(3))
        tree.set()
        outs = [torch.empty(B, T, H, d, dtype=dtype, device="cuda") for _ in range(L)]
        for layer in range(L):
            tree.attention(layer, qs[layer], ks[layer], vs[layer], outs[layer])
        take = (T, 4)
        path = torch.arange(T, dtype=torch.int32, device="cuda").repeat(B, 1)
        tree.commit(ks, vs, path, _ints(take))
        tree.advance()
        for i in range(T):
            for layer in range(L):
                o = torch.empty(B, H, d, dtype=dtype, device="cuda")
                a.decode_step(layer, qs[layer][:, i].contiguous(), ks[layer][:, i].contiguous(),
                              vs[layer][:, i].contiguous(), o)
                for r in range(B):
                    err = float((o[r].double() - outs[layer][r, i].double()).abs().max())
                    assert i >= take[r] or err <= tol, (step, i, layer, r, err)
            a.advance()
            if i == 3:  # the second sequence stops here: keep its rings and counter
                saved = [[(a.cache_view(layer, w, 1, h).clone(), layer, w, h) for h in range(H)]
                         for layer in range(L) for w in "kv"]
                t_saved = a.ring()[0][1]
        # sequence 0 took all T; sequence 1 took 4: compare each with the decode path
        for layer in range(L):
            for h in range(H):
                for w in "kv":
                    x, y = a.cache_view(layer, w, 0, h), b.cache_view(layer, w, 0, h)
                    held = plens[0] + min(a.ring()[0][0], W)
                    assert torch.equal(x[:held], y[:held])
        for group in saved:
            for x, layer, w, h in group:
                held = plens[1] + min(t_saved, W)
                assert torch.equal(x[:held], b.cache_view(layer, w, 1, h)[:held])
                a.cache_view(layer, w, 1, h).copy_(b.cache_view(layer, w, 1, h))
        assert b.ring()[0][0] == a.ring()[0][0] and b.ring()[0][1] == t_saved
        # rebuild the decode side at the tree side's counters for the next step
        na = rswa.State(B, L, H, d, W, plens, dtype=dtype, n_generated=b.ring()[0])
        for layer in range(L):
            na.k_cache[layer].copy_(b.k_cache[layer])
            na.v_cache[layer].copy_(b.v_cache[layer])
        if rope:
            na.set_rope(rope)
        if swa:
            na.set_attention(rswa.RSWA_ATTN_STANDARD_SWA)
        a = na
    assert a.check() == 0 and b.check() == 0


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
def test_standard_window_matches_the_definition(dtype, d):
    rswa = _rswa()
    c = Case(dtype, d, 2, 70, (300, 40, 71), (20, 90, 0), 13)
    c.st.set_attention(rswa.RSWA_ATTN_STANDARD_SWA)
    c.check(c.run(), swa=True)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F32, 64)])
@pytest.mark.parametrize("swa", [False, True])
def test_wide_trees(dtype, d, swa):
    """More drafts than one group of rows takes, in some sequences only: counts around the
    group's edge, a branch that crosses it, and bad values in the first group's rows."""
    rswa = _rswa()
    T, n = 100, (100, 65, 64, 1, 0)
    rng = np.random.default_rng(12)
    parents = [ref.random_parents(rng, T, reach=40) for _ in n]
    c = Case(dtype, d, 2, 40, (300, 20, 77, 0, 50), (50, 3, 200, 39, 1), T, n=n, parents=parents)
    if swa:
        c.st.set_attention(rswa.RSWA_ATTN_STANDARD_SWA)
    rows = (0, 1, 31, 32, 62, 63, 64, 65, 98, 99)
    clean = c.run()
    c.check(clean, swa=swa, rows=rows)
    c.v[0, 10, :, 3] = float("nan")
    out = c.run()
    sees = [i for i in range(T) if 10 in ref.path_of(parents[0], i)[-40:]]
    blind = [i for i in range(T) if i not in sees]
    assert torch.equal(out[0, blind], clean[0, blind]) and torch.equal(out[1:], clean[1:])
    assert bool(out[0, sees, :, 3].isnan().all())
    others = [e for e in range(d) if e != 3]
    assert torch.equal(out[0, sees][..., others], clean[0, sees][..., others])


@pytest.mark.parametrize("dtype,d", KINDS)
@pytest.mark.parametrize("T", [68, 72, 80, 96, 127])
def test_trees_a_little_wider_than_a_group(dtype, d, T):
    """A few rows past 64 drafts, chains among them, values and keys unseen by some not finite."""
    rng = np.random.default_rng(T)
    n = (T, 66, 64, 3)
    parents = [[i - 1 for i in range(T)]] + [ref.random_parents(rng, T, reach=50) for _ in n[1:]]
    c = Case(dtype, d, 2, 100, (61, 189, 0, 130), (100, 7, 300, 0), T, n=n, parents=parents)
    rows = (0, 1, 15, 16, 31, 62, 63, 64, 65, 66, 67, 70, 71, 79, 80, 95, 126)
    clean = c.run()
    c.check(clean, rows=rows)
    # the last drafts of the first sequence: seen by themselves and each other alone
    c.k[0, T - 2:, :, 1] = float("inf")
    c.v[0, T - 2:, :, 2] = -float("inf")
    out = c.run()
    assert torch.equal(out[0, :T - 2], clean[0, :T - 2]) and torch.equal(out[1:], clean[1:])


@pytest.mark.parametrize("dtype,d", KINDS)
@pytest.mark.parametrize("rope", [1, 2])
def test_wide_trees_turn_with_rope(dtype, d, rope):
    """Every node of a 100-node tree under RoPE gives what a tree of its path alone gives."""
    T, plens, t = 100, (140, 9), (20, 3)
    c = Case(dtype, d, 2, 16, plens, t, T, n=(T, 70))
    c.st.set_rope(rope)
    out = c.run()
    for b, i in ((0, 99), (0, 64), (0, 63), (1, 69), (1, 5)):
        path = ref.path_of(c.parents[b], i)
        m = len(path)
        one = c.st.tree(m)
        q, k, v = (torch.zeros(2, m, 2, d, dtype=dtype) for _ in range(3))
        for x, y in ((q, c.q), (k, c.k), (v, c.v)):
            x[b] = y[b, path]
        n = [m if x == b else 0 for x in range(2)]
        got = torch.zeros(2, m, 2, d, dtype=dtype, device="cuda")
        one.set(None, _ints(n))
        one.attention(0, q.cuda(), k.cuda(), v.cuda(), got)
        # the same sums in another order, and another subtracted maximum
        tol = 2e-2 if dtype == BF else 1e-5
        assert float((got[b, -1].cpu().double() - out[b, i].double()).abs().max()) <= tol
    assert c.st.check() == 0


def _rotated(x, pos, theta):
    """x [H, d] turned at position pos (rotate-half), in 64 bits."""
    half = x.shape[-1] // 2
    a = pos * theta ** (-2.0 * torch.arange(half, dtype=torch.float64) / x.shape[-1])
    x0, x1 = x[..., :half].double(), x[..., half:].double()
    return torch.cat([x0 * a.cos() - x1 * a.sin(), x1 * a.cos() + x0 * a.sin()], -1)


@pytest.mark.parametrize("dtype,d", KINDS)
@pytest.mark.parametrize("T", [5, 16, 20])
@pytest.mark.parametrize("rope", [1, 2])
def test_short_rings_turn_with_rope(dtype, d, T, rope):
    """More rings than SMs, each of a few tiles at most, so a CTA turns one ring's queries
    after another's while little else holds it up.  The queries and drafted keys that the
    reference attends with are turned in 64 bits and rounded to the element type, as the
    call documents.  The kernel turns them in fp32: sines and cosines to 2 steps, two products
    and a sum, so 2^-21 of the vector's length at most, on q and on k.  In bf16 a component
    within that of a rounding's border (1 in 2^14 of them; more than 4 along a path of 20 in
    no case of 10^8) falls to the other side, one step (eps) away.  An error x of a score
    changes the output by up to 2 x of the mass."""
    rswa = _rswa()
    B, H, W, theta = 100, 4, 16, 10000.0
    rng = np.random.default_rng(T)
    plens = [int(x) for x in rng.integers(0, 100, B)]
    t = [int(x) for x in rng.integers(0, 40, B)]
    n = [int(x) for x in rng.integers(0, T + 1, B)]
    c = Case(dtype, d, H, W, plens, t, T, n=n)
    c.st.set_rope(rope, theta)
    out = c.run()
    assert torch.equal(out, c.run())
    m = c.model
    for b in range(0, B, 3):
        for i in {0, n[b] // 2, n[b] - 1}:
            if not 0 <= i < n[b]:
                continue
            path = ref.path_of(c.parents[b], i)

            def pos(e):
                return plens[b] + ((t[b] + e) % W if rope == 2 else t[b] + e)

            ks = [_rotated(c.k[b, x], pos(e), theta).to(dtype) for e, x in enumerate(path)]
            qt = _rotated(c.q[b, i], pos(len(path) - 1), theta).to(dtype)
            for h in range(H):
                k, v = m.entries(b, h, ks, [c.v[b, x] for x in path])
                o, mass = ref.attend(qt[h], k, v, c.scale)
                qh = qt[h].double()
                x = 2.0 ** -20 * float(qh.norm() * k.norm(dim=1).max()) * c.scale
                if dtype == BF:
                    x += 4 * torch.finfo(BF).eps * float(qh.abs().max() * k.abs().max()) * c.scale
                lim = ref.tolerance(o, mass, dtype) + 2 * x * mass
                err = (out[b, i, h].double() - o).abs()
                assert bool((err <= lim).all()), (b, i, h, float((err / lim).max()))


@pytest.mark.parametrize("dtype,d", KINDS)
def test_commit_writes_the_path_and_nothing_else(dtype, d):
    L, H, W, plens, t, T = 3, 2, 6, (5, 9, 0, 4), (2, 11, 6, 30), 10
    c = Case(dtype, d, H, W, plens, t, T, layers=L)
    c.parents = [[i - 1 for i in range(T)], [-1, -1, 0, 2, 1, 4, 5, 5, 7, 8], [-1] * T,
                 [i - 1 for i in range(T)]]
    paths = [[0, 1, 2], [1, 4, 5, 7, 8, 9], [], list(range(T))]  # the last is longer than W
    before = [[x.clone() for x in c.st.k_cache], [x.clone() for x in c.st.v_cache]]
    ks, vs = ([c.model.draw(len(plens), T, H, d).cuda() for _ in range(L)] for _ in range(2))
    path = torch.zeros(len(plens), T, dtype=torch.int32)
    for b, p in enumerate(paths):
        path[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
    c.tree.set(_ints(c.parents))
    c.tree.commit(ks, vs, path.cuda(), _ints([len(p) for p in paths]))
    base = 0
    for b, p in enumerate(paths):
        size = plens[b] + W
        for i, node in list(enumerate(p)):
            for layer in range(L):
                for h in range(H):
                    row = base * H + h * size + plens[b] + (t[b] + i) % W
                    for buf, src in ((before[0], ks), (before[1], vs)):
                        buf[layer].view(-1, d)[row] = src[layer][b, node, h]
        base += size
    same = [torch.equal(x.view(torch.uint8), y.view(torch.uint8))
            for x, y in zip(c.st.k_cache + c.st.v_cache, before[0] + before[1])]
    assert all(same)
    assert c.st.ring()[0] == list(t)
    c.tree.advance()
    assert c.st.ring()[0] == [x + len(p) for x, p in zip(t, paths)]
    c.tree.advance()  # counted once
    assert c.st.ring()[0] == [x + len(p) for x, p in zip(t, paths)]
    assert c.st.check() == 0


def test_commit_into_many_layers():
    """More layers than one launch takes, every one with its own drafts."""
    rswa = _rswa()
    L, H, d, W, P, T, t = 67, 1, 64, 5, 3, 4, 6
    st = rswa.State(1, L, H, d, W, (P,), dtype=BF, n_generated=(t,))
    for x in st.k_cache + st.v_cache:
        x.fill_(1.0)
    g = torch.Generator(device="cuda").manual_seed(2)
    ks, vs = ([torch.randn(1, T, H, d, generator=g, device="cuda").to(BF) for _ in range(L)]
              for _ in range(2))
    tree = st.tree(T)
    tree.set()
    tree.commit(ks, vs, _ints([[0, 1, 2, 0]]), _ints([3]))
    tree.advance()
    assert st.check() == 0 and st.ring()[0] == [t + 3]
    for layer in range(L):
        for w, src in (("k", ks), ("v", vs)):
            want = torch.ones(P + W, d, dtype=BF, device="cuda")
            for i in range(3):
                want[P + (t + i) % W] = src[layer][0, i, 0]
            assert torch.equal(st.cache_view(layer, w, 0, 0), want)


def test_bad_trees_and_paths_are_refused_sequence_by_sequence():
    rswa = _rswa()
    T, W = 6, 8
    c = Case(BF, 128, 2, W, (20, 20, 20, 20, 20), (3, 3, 3, 3, 3), T)
    good = [-1, 0, 1, 1, 3, 0]
    # own parent, a later parent, below -1, a count above T
    c.parents = [good, [-1, 1, 0, 0, 0, 0], [-1, 0, 5, 0, 0, 0], [-2, 0, 0, 0, 0, 0], good]
    c.tree.set(_ints(c.parents), _ints([T, T, T, T, T + 1]))
    out = torch.full((5, T, 2, 128), 7.0, dtype=BF, device="cuda")
    c.tree.attention(0, c.q.cuda(), c.k.cuda(), c.v.cuda(), out)
    assert c.st.check() == rswa.RSWA_EDEVICE
    assert c.st.check() == 0
    assert bool((out[1:] == 7.0).all()) and bool((out[0] != 7.0).any())
    # paths: not a chain, not from a first node, a node out of range, too long, of a refused tree
    c.tree.set(_ints([good] * 5), _ints([T, T, T, T, 4]))
    before = [x.clone() for x in c.st.k_cache + c.st.v_cache]
    paths = [[0, 1, 4, 0, 0, 0], [1, 3, 0, 0, 0, 0], [0, 6, 0, 0, 0, 0], [0] * T, [0, 1, 3, 4, 0, 0]]
    c.tree.commit([c.k.cuda()], [c.v.cuda()], _ints(paths), _ints([3, 2, 2, T + 1, 4]))
    assert c.st.check() == rswa.RSWA_EDEVICE
    for x, y in zip(before, c.st.k_cache + c.st.v_cache):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    c.tree.advance()
    assert c.st.ring()[0] == [3] * 5
    # padding behind the drafts is not looked at
    c.tree.set(_ints([good[:3] + [99, -7, 5]] * 5), _ints([3] * 5))
    assert c.st.check() == 0


def test_tree_step_in_a_graph():
    """set, attention, commit and advance captured once and replayed over new inputs."""
    T, W, L, H, d, plens, t = 5, 7, 2, 2, 128, (140, 30), (4, 9)
    c, e = (Case(BF, d, H, W, plens, t, T, layers=L, seed=9) for _ in range(2))
    static = {"parent": _ints(c.parents), "n": _ints([T, T]), "path": _ints([[0] * T] * 2),
              "len": _ints([0, 0])}
    qs, ks, vs = ([torch.zeros(2, T, H, d, dtype=BF, device="cuda") for _ in range(L)]
                  for _ in range(3))
    outs = [torch.zeros_like(x) for x in qs]

    def step(x):
        x.tree.set(static["parent"], static["n"])
        for layer in range(L):
            x.tree.attention(layer, qs[layer], ks[layer], vs[layer], outs[layer])
        x.tree.commit(ks, vs, static["path"], static["len"])
        x.tree.advance()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(c)  # warm-up on zeros: nothing accepted
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(c)
    rng = np.random.default_rng(2)
    for _ in range(5):
        parents = [ref.random_parents(rng, T) for _ in range(2)]
        paths = [ref.path_of(p, int(rng.integers(0, T))) for p in parents]
        static["parent"].copy_(_ints(parents))
        static["path"].copy_(_ints([p + [0] * (T - len(p)) for p in paths]))
        static["len"].copy_(_ints([len(p) for p in paths]))
        for x in qs + ks + vs:
            x.copy_(c.model.draw(2, T, H, d))
        graph.replay()
        got = [x.clone() for x in outs]
        step(e)
        for x, y in zip(got, outs):
            assert torch.equal(x, y)
        for x, y in zip(c.st.k_cache + c.st.v_cache, e.st.k_cache + e.st.v_cache):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
        assert c.st.ring() == e.st.ring()
    assert c.st.check() == 0 and e.st.check() == 0


def test_two_trees_on_two_streams():
    """Two states, each with its tree, stepped at the same time on streams of their own."""
    cases = [Case(BF, 128, 4, 64, (3000, 500), (70, 9), 31, seed=s) for s in (21, 22)]
    want = [c.run() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    ins = [(c.q.cuda(), c.k.cuda(), c.v.cuda(), _ints(c.parents)) for c in cases]
    outs = [torch.full_like(i[0], 7.0) for i in ins]
    torch.cuda.synchronize()
    for _ in range(4):
        for c, s, i, o in zip(cases, streams, ins, outs):
            c.tree.set(i[3], None, stream=s)
            c.tree.attention(0, i[0], i[1], i[2], o, stream=s)
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert torch.equal(w, o.cpu())


def test_repeats_are_equal_bit_for_bit():
    c = Case(BF, 128, 3, 128, (4000, 300), (200, 50), 47)
    first = c.run()
    for _ in range(3):
        assert torch.equal(first, c.run())


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
def test_tree_over_a_pool(dtype, d):
    """Requests placed anywhere in a pool, other requests' slots holding NaN."""
    rswa = _rswa()
    H, W, plens, t, T = 2, 9, (33, 140), (4, 12), 6
    pool = rswa.TokenPool(600, 1, H, d, W, dtype=dtype)
    pool.k_cache[0].fill_(float("nan"))
    pool.v_cache[0].fill_(float("nan"))
    pool.alloc(50)
    bases = [pool.alloc(p) for p in plens][::-1]
    bases = [pool.alloc(plens[0]), bases[0]]
    c = Case(dtype, d, H, W, plens, t, T)
    st = pool.state(plens, bases, n_generated=t)
    c.model.fill(st)
    c.st, c.tree = st, st.tree(T)
    c.check(c.run())


def test_refusals():
    rswa = _rswa()
    c = Case(BF, 128, 2, 8, (20,), (3,), 4)
    q, k, v = c.q.cuda(), c.k.cuda(), c.v.cuda()
    out = torch.empty_like(q)
    for T in (0, -1, rswa.RSWA_TREE_MAX + 1):
        with pytest.raises(rswa.RswaError):
            c.st.tree(T)
    with pytest.raises(rswa.RswaError) as e:
        rswa.rswa_tree_create(c.st.handle, 4, c.tree.workspace, 16)
    assert e.value.status == rswa.RSWA_ENOMEM
    bad = [(1, q, k, v, out), (-1, q, k, v, out), (0, q[:, :2], k, v, out),
           (0, q.float(), k, v, out), (0, q.cpu(), k, v, out),
           (0, q.transpose(1, 2).contiguous().transpose(1, 2), k, v, out),
           (0, q, k, v, q), (0, q, k, v, k), (0, q, k, v, v)]
    for args in bad:
        with pytest.raises(rswa.RswaError) as e:
            c.tree.attention(*args)
        assert e.value.status == rswa.RSWA_EINVAL
    with pytest.raises(rswa.RswaError):
        rswa.rswa_tree_attention(c.tree.handle, 0, q.data_ptr() + 2, k, v, out)
    with pytest.raises(rswa.RswaError):
        c.tree.set(torch.zeros(1, 4, dtype=torch.int64, device="cuda"))
    with pytest.raises(rswa.RswaError):
        c.tree.commit([k, k], [v, v], _ints([[0] * 4]), _ints([1]))
    fresh = rswa.State(1, 1, 2, 128, 8, [20], dtype=BF)
    tree = fresh.tree(4)
    tree.set()
    with pytest.raises(rswa.RswaError) as e:
        tree.attention(0, q, k, v, out)
    assert e.value.status == rswa.RSWA_ESTATE
    with pytest.raises(rswa.RswaError) as e:
        tree.commit([k], [v], _ints([[0] * 4]), _ints([1]))
    assert e.value.status == rswa.RSWA_ESTATE
    # before any rswa_tree_set nothing is drafted
    out.fill_(7.0)
    c.tree.attention(0, q, k, v, out)
    assert bool((out == 7.0).all())
