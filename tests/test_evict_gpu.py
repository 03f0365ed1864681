"""Scored decode steps and eviction by accumulated weight, against the definition in 64
bits, and a run of prefill, scored decoding, eviction and draft verification together."""
import numpy as np
import pytest
import torch

import tree_reference as ref
from helpers import F32_TOL, f64, tol_for

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
KINDS = [(BF, 128), (BF, 64), (F32, 128), (F32, 64)]


def _rswa():
    from ring_sliding_window_b200 import rswa
    return rswa


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _bits(t):
    return t.contiguous().view(torch.uint8)


def _weights(m, b, h, q, scale, swa=False):
    """Softmax weights of the newest token over (prompt entries seen, generated seen)."""
    k = torch.stack([x[h] for x in m.gk[b]][-m.W:])
    pk = m.pk[b][:, h]
    cut = min(len(pk), max(0, m.plens[b] + len(m.gk[b]) - m.W)) if swa else 0
    s = torch.cat([pk[cut:], k]).double() @ q.double() * scale
    w = torch.softmax(s, 0)
    return cut, w[:len(pk) - cut], w[len(pk) - cut:]


@pytest.mark.parametrize("dtype,d", KINDS)
@pytest.mark.parametrize("split", ["streamk", "cluster"])
@pytest.mark.parametrize("in_place", [False, True])
def test_scored_steps_accumulate_the_softmax_weights(dtype, d, split, in_place, monkeypatch):
    """2 W + 3 steps across two ring wraps.  A weight is at most 1; its fp32 score, exponential
    and sum are good to some 1e-6, and each of the n additions rounds by half a step of a sum
    of at most n: n * (2e-6 + n 2^-24)."""
    rswa = _rswa()
    monkeypatch.setenv("RSWA_DECODE_SPLIT", split)
    H, W, plens = 2, 6, (130, 0, 2500)
    B = len(plens)
    m = ref.Model(plens, W, H, d, dtype, seed=2)
    st = rswa.State(B, 1, H, d, W, plens, dtype=dtype, n_generated=[0] * B)
    twin = rswa.State(B, 1, H, d, W, plens, dtype=dtype, n_generated=[0] * B)
    m.fill(st)
    m.fill(twin)
    a = st.score_buffer().fill_(float("nan"))
    want = {}
    for b, P in enumerate(plens):
        for h in range(H):
            st.score_view(a, b, h)[:P] = 0.25
            want[b, h] = np.full(P + W, np.nan)
            want[b, h][:P] = 0.25
    c, scratch = (a if in_place else a.clone()), torch.empty_like(a)
    n = 2 * W + 3
    for step in range(n):
        q, kn, vn = (m.draw(B, H, d) for _ in range(3))
        out, out2 = (torch.empty(B, H, d, dtype=dtype, device="cuda") for _ in range(2))
        st.decode_step_scored(0, q.cuda(), kn.cuda(), vn.cuda(), out, a, c, scratch)
        twin.decode_step(0, q.cuda(), kn.cuda(), vn.cuda(), out2)
        assert torch.equal(out, out2)  # the same attention, bit for bit
        a, c = c, a
        for b, P in enumerate(plens):
            m.gk[b].append(kn[b])
            m.gv[b].append(vn[b])
            t = len(m.gk[b])
            for h in range(H):
                _, wp, wg = _weights(m, b, h, q[b, h], d ** -0.5)
                want[b, h][:P] += wp.numpy()
                want[b, h][P + (t - 1) % W] = 0.0
                for i, w in enumerate(wg.tolist()):
                    want[b, h][P + (t - len(wg) + i) % W] += w
                got = f64(st.score_view(a, b, h))
                held = P + min(t, W)
                assert np.all(np.isnan(got[held:]))
                assert np.max(np.abs(got[:held] - want[b, h][:held])) <= n * (2e-6 + n * 2.0 ** -24)
        st.advance()
        twin.advance()
    for x, y in zip(st.k_cache + st.v_cache, twin.k_cache + twin.v_cache):
        assert torch.equal(_bits(x), _bits(y))
    assert st.check() == 0


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
def test_scored_steps_in_the_standard_window(dtype, d):
    rswa = _rswa()
    H, W, plens = 2, 40, (100, 10)
    m = ref.Model(plens, W, H, d, dtype, seed=3).generate((7, 60))
    st = rswa.State(2, 1, H, d, W, plens, dtype=dtype, n_generated=m.t)
    st.set_attention(rswa.RSWA_ATTN_STANDARD_SWA)
    m.fill(st)
    before = torch.rand(rswa.rswa_score_bytes(st.handle) // 4, device="cuda")
    after, scratch = torch.full_like(before, float("nan")), torch.empty_like(before)
    q, kn, vn = (m.draw(2, H, d) for _ in range(3))
    out = torch.empty(2, H, d, dtype=dtype, device="cuda")
    st.decode_step_scored(0, q.cuda(), kn.cuda(), vn.cuda(), out, before, after, scratch)
    for b, P in enumerate(plens):
        m.gk[b].append(kn[b])
        m.gv[b].append(vn[b])
        t = len(m.gk[b])
        for h in range(H):
            cut, wp, wg = _weights(m, b, h, q[b, h], d ** -0.5, swa=True)
            want = f64(st.score_view(before, b, h)).copy()
            want[cut:P] += wp.numpy()
            want[P + (t - 1) % W] = 0.0
            for i, w in enumerate(wg.tolist()):
                want[P + (t - len(wg) + i) % W] += w
            held = P + min(t, W)
            assert np.max(np.abs(f64(st.score_view(after, b, h))[:held] - want[:held])) <= 4e-6
            assert np.all(np.isnan(f64(st.score_view(after, b, h))[held:]))


@pytest.mark.parametrize("dtype,d", KINDS)
@pytest.mark.parametrize("split", ["streamk", "cluster"])
@pytest.mark.parametrize("rope", [0, 1, 2])
def test_scored_steps_with_rope_over_a_pool(dtype, d, split, rope, monkeypatch):
    """Requests placed out of order in a pool whose other slots, and their scores, hold NaN.  The
    weights are those of the keys that the step left in the cache, turned there, and of the
    query turned in 64 bits; the kernel turns it in fp32, 2^-21 of its length off at most, which
    moves a score by that times the longest key, and a weight (at most 1) by twice as much."""
    rswa = _rswa()
    monkeypatch.setenv("RSWA_DECODE_SPLIT", split)
    H, W, plens, t, steps, theta = 2, 6, (130, 7, 1500), (0, 11, 4), 15, 10000.0
    B = len(plens)
    pool = rswa.TokenPool(2400, 1, H, d, W, dtype=dtype)
    for x in pool.k_cache + pool.v_cache:
        x.fill_(float("nan"))
    pool.alloc(20)
    bases = {p: pool.alloc(p) for p in (7, 1500, 130)}
    st = pool.state(plens, [bases[p] for p in plens], n_generated=t)
    twin_pool = rswa.TokenPool(2400, 1, H, d, W, dtype=dtype)
    m = ref.Model(plens, W, H, d, dtype, seed=12).generate(t)
    m.fill(st)
    for x, y in zip(twin_pool.k_cache + twin_pool.v_cache, pool.k_cache + pool.v_cache):
        x.copy_(y)
    twin = twin_pool.state(plens, [bases[p] for p in plens], n_generated=t)
    for x in (st, twin):
        x.set_rope(rope, theta)
    score, scratch = st.score_buffer().fill_(float("nan")), st.score_buffer()
    want, mine = {}, torch.zeros(score.numel(), dtype=torch.bool, device="cuda")
    for b, P in enumerate(plens):
        for h in range(H):
            held = P + min(t[b], W)
            st.score_view(score, b, h)[:held] = 0.5
            st.score_view(mine, b, h)[:] = True
            want[b, h] = np.full(P + W, 0.5)
    slack = 0.0
    for step in range(steps):
        q, kn, vn = (m.draw(B, H, d).cuda() for _ in range(3))
        out, out2 = torch.empty_like(q), torch.empty_like(q)
        st.decode_step_scored(0, q, kn, vn, out, score, score, scratch)
        twin.decode_step(0, q, kn, vn, out2)
        assert torch.equal(out, out2)
        for b, P in enumerate(plens):
            now = t[b] + step
            held, fresh = P + min(now + 1, W), P + now % W
            pos = P + (now % W if rope == 2 else now)
            for h in range(H):
                k = st.cache_view(0, "k", b, h)[:held].double().cpu()
                x = q[b, h].double().cpu()
                if rope:
                    half = d // 2
                    angle = pos * theta ** (-2.0 * torch.arange(half, dtype=torch.float64) / d)
                    x = torch.cat([x[:half] * angle.cos() - x[half:] * angle.sin(),
                                   x[half:] * angle.cos() + x[:half] * angle.sin()])
                    slack = max(slack, 2.0 ** -20 * float(x.norm() * k.norm(dim=1).max()) * d ** -0.5)
                want[b, h][fresh] = 0.0
                want[b, h][:held] += torch.softmax(k @ x * d ** -0.5, 0).numpy()
                got = f64(st.score_view(score, b, h))
                lim = (step + 1) * (2e-6 + (step + 2) * 2.0 ** -24 + slack)
                assert np.max(np.abs(got[:held] - want[b, h][:held])) <= lim
                assert np.all(np.isnan(got[held:]))
        assert bool(score[~mine].isnan().all())
        st.advance()
        twin.advance()
    for x, y in zip(pool.k_cache + pool.v_cache, twin_pool.k_cache + twin_pool.v_cache):
        assert torch.equal(_bits(x), _bits(y))
    assert st.check() == 0


def _fill_random(st, dtype, layers, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    for layer in range(layers):
        for buf in (st.k_cache[layer], st.v_cache[layer]):
            buf.copy_(torch.randn(buf.numel(), generator=g, device="cuda").to(dtype))


def _check_evicted(src, dst, layer, score, dst_score, kept, first, last, t, H):
    W, base = src.W, 0
    for b, (P, K) in enumerate(zip(src.prefill_lens, dst.prefill_lens)):
        ring = min(t[b], W)
        for h in range(H):
            want = ref.kept_slots(f64(src.score_view(score, b, h)[:P]), K, first, last)
            got = kept[base + h * K:base + (h + 1) * K].tolist()
            assert got == want, (b, h)
            rows = torch.tensor(want + list(range(P, P + ring)), device="cuda", dtype=torch.int64)
            for w in "kv":
                x, y = src.cache_view(layer, w, b, h)[rows], dst.cache_view(layer, w, b, h)
                assert torch.equal(_bits(x), _bits(y[:K + ring]))
                assert bool((y[K + ring:] == 5.0).all())
            s, r = src.score_view(score, b, h)[rows], dst.score_view(dst_score, b, h)
            assert torch.equal(_bits(s), _bits(r[:K + ring]))
            assert bool((r[K + ring:] == 5.0).all())
        base += H * K


@pytest.mark.parametrize("dtype,d", KINDS)
@pytest.mark.parametrize("plens,keep,first,last,t,W", [
    ((1,), (1,), 0, 0, (0,), 3),
    ((9, 0, 40), (4, 0, 40), 1, 2, (2, 7, 3), 5),         # some, nothing to keep, everything
    ((300, 1088, 77), (0, 333, 76), 0, 0, (0, 130, 9), 128),
    ((5000, 33), (2500, 33), 64, 256, (200, 5), 17),       # protection covers a whole prompt
    ((513, 4097), (512, 1), 0, 1, (6, 6), 6),
])
def test_evict_keeps_the_highest_scores(dtype, d, plens, keep, first, last, t, W):
    rswa = _rswa()
    if any(min(first + last, p) > k for p, k in zip(plens, keep)):
        pytest.fail("case breaks the call's contract")
    H, L = 3, 2
    src = rswa.State(len(plens), L, H, d, W, plens, dtype=dtype, n_generated=t)
    dst = rswa.State(len(plens), L, H, d, W, keep, dtype=dtype)
    _fill_random(src, dtype, L, 4)
    for buf in dst.k_cache + dst.v_cache:
        buf.fill_(5.0)
    for layer in range(L):
        score = torch.rand(src.score_buffer().numel(), device="cuda").pow(4)
        score[torch.rand_like(score) < 0.4] = 0.0     # many ties
        score[torch.rand_like(score) < 0.05] = 0.5
        out = torch.full((rswa.rswa_score_bytes(dst.handle) // 4,), 5.0, device="cuda")
        kept = src.evict_into(dst, layer, score, first, last, out)
        _check_evicted(src, dst, layer, score, out, kept, first, last, t, H)
    assert dst.ring()[0] == list(t)
    dst.advance()
    dst.reset_ring()
    assert dst.ring()[0] == list(t)


@pytest.mark.parametrize("plens,t", [((40,), (5,)), ((0,), (9,)), ((0, 300, 1), (0, 2, 30))])
def test_evict_that_keeps_no_prompt_entry(plens, t):
    """The ring alone moves; the list of kept slots is empty and has no address."""
    rswa = _rswa()
    H, W, d, B = 2, 7, 64, len(plens)
    src = rswa.State(B, 1, H, d, W, plens, dtype=F32, n_generated=t)
    dst = rswa.State(B, 1, H, d, W, (0,) * B, dtype=F32)
    _fill_random(src, F32, 1, 6)
    for buf in dst.k_cache + dst.v_cache:
        buf.fill_(5.0)
    score = torch.rand(src.score_buffer().numel(), device="cuda")
    out = torch.full((rswa.rswa_score_bytes(dst.handle) // 4,), 5.0, device="cuda")
    kept = src.evict_into(dst, 0, score, 0, 0, out)
    assert kept.numel() == 0
    _check_evicted(src, dst, 0, score, out, kept, 0, 0, t, H)
    assert dst.ring()[0] == list(t)
    # a list that is not empty needs its address
    one = rswa.State(B, 1, H, d, W, tuple(min(1, p) for p in plens), dtype=F32)
    if sum(plens) > 0:
        with pytest.raises(rswa.RswaError) as e:
            rswa.rswa_evict(src.handle, one.handle, 0, score, 0, 0, None, None)
        assert e.value.status == rswa.RSWA_EINVAL


def test_evict_orders_every_float():
    """Signed zeros tie, infinities and denormals rank by value, NaN ranks last, and
    protected slots stay even at NaN."""
    rswa = _rswa()
    special = [0.0, -0.0, float("inf"), -float("inf"), float("nan"), -float("nan"), 1e-45, -1e-45,
               3.4e38, -3.4e38, 1.0, -1.0]
    rng = np.random.default_rng(0)
    P, W, H = 600, 4, 2
    for keep in (3, 60, 300, 597):
        src = rswa.State(1, 1, H, 64, W, (P,), dtype=F32, n_generated=(2,))
        dst = rswa.State(1, 1, H, 64, W, (keep,), dtype=F32)
        _fill_random(src, F32, 1, 1)
        for buf in dst.k_cache + dst.v_cache:
            buf.fill_(5.0)
        score = torch.tensor(rng.choice(special, H * (P + W)), dtype=F32, device="cuda")
        score[0] = score[P - 1] = float("nan")
        out = torch.full((H * (keep + W),), 5.0, device="cuda")
        kept = src.evict_into(dst, 0, score, 1, 2, out)
        _check_evicted(src, dst, 0, score, out, kept, 1, 2, (2,), H)


@pytest.mark.parametrize("P", [49151, 49152, 49157, 120001])
def test_evict_from_long_prompts(P):
    """Prompts around and beyond what a CTA's shared memory holds: many values, and ties."""
    rswa = _rswa()
    H, W, first, last = 2, 3, 5, 70
    for keep in (100, P // 3, P - 1):
        src = rswa.State(1, 1, H, 64, W, (P,), dtype=BF, n_generated=(2,))
        dst = rswa.State(1, 1, H, 64, W, (keep,), dtype=BF)
        _fill_random(src, BF, 1, 1)
        for kind in range(3):
            score = torch.rand(src.score_buffer().numel(), device="cuda").pow(6) - 0.2
            if kind == 1:
                score = (score * 8).round() / 8
            if kind == 2:
                score[torch.rand_like(score) < 0.9] = 0.0
            kept = src.evict_into(dst, 0, score, first, last).view(H, keep)
            for h in range(H):
                rank = src.score_view(score, 0, h)[:P].clone()
                rank[:first] = rank[P - last:] = float("inf")
                order = torch.sort(rank, descending=True, stable=True).indices[:keep]
                want = torch.sort(order).values
                assert torch.equal(kept[h].long(), want)
                assert torch.equal(_bits(dst.cache_view(0, "k", 0, h)[:keep]),
                                   _bits(src.cache_view(0, "k", 0, h)[want]))


def test_all_scores_equal_keeps_the_first_slots():
    rswa = _rswa()
    P, keep, H = 20000, 7777, 2
    src = rswa.State(1, 1, H, 128, 8, (P,), dtype=BF, n_generated=(0,))
    dst = rswa.State(1, 1, H, 128, 8, (keep,), dtype=BF)
    _fill_random(src, BF, 1, 1)
    kept = src.evict_into(dst, 0, src.score_buffer())
    assert torch.equal(kept.view(H, keep).cpu(), torch.arange(keep, dtype=torch.int32).repeat(H, 1))


@pytest.mark.parametrize("rope", [1, 2])
@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
def test_positions_survive_an_eviction(rope, dtype, d):
    """Keeping every entry changes nothing, so decoding on with RoPE gives the same bits; keeping
    some gives attention over those, with the uncut prompt's positions.  A second eviction of
    the result still counts from the first prompt."""
    rswa = _rswa()
    H, W, P, t = 2, 5, 60, 7
    src = rswa.State(1, 1, H, d, W, (P,), dtype=dtype, n_generated=(t,))
    src.set_rope(rope)
    _fill_random(src, dtype, 1, 8)
    g = torch.Generator(device="cuda").manual_seed(1)
    score = torch.rand(H * (P + W), generator=g, device="cuda")
    part = rswa.State(1, 1, H, d, W, (40,), dtype=dtype)
    part_score = torch.zeros(H * (40 + W), device="cuda")
    kept = src.evict_into(part, 0, score, dst_score=part_score).view(H, 40).long()
    again = rswa.State(1, 1, H, d, W, (40,), dtype=dtype)
    part.evict_into(again, 0, part_score)
    whole = rswa.State(1, 1, H, d, W, (P,), dtype=dtype)
    src.evict_into(whole, 0, score)
    for step in range(2 * W):
        q, kn, vn = (torch.randn(1, H, d, generator=g, device="cuda").to(dtype) for _ in range(3))
        outs = []
        for st in (src, whole, part, again):
            out = torch.empty_like(q)
            st.decode_step(0, q, kn, vn, out)
            outs.append(out)
        assert torch.equal(outs[0], outs[1])
        assert torch.equal(outs[2], outs[3])
        new = (t + step) % W
        for h in range(H):
            assert torch.equal(src.cache_view(0, "k", 0, h)[P + new],
                               part.cache_view(0, "k", 0, h)[40 + new])
        for st in (src, whole, part, again):
            st.advance()
    for h in range(H):
        assert torch.equal(part.cache_view(0, "k", 0, h)[:40], src.cache_view(0, "k", 0, h)[kept[h]])


def test_evict_inside_a_pool_and_out_of_it():
    rswa = _rswa()
    H, W, d, P, K = 2, 4, 128, 50, 20
    pool = rswa.TokenPool(200, 1, H, d, W, dtype=BF)
    _fill_random(pool, BF, 1, 3)
    big = pool.alloc(P)
    src = pool.state((P,), (big,), n_generated=(9,))
    small = pool.alloc(K)
    dst = pool.state((K,), (small,))
    score = torch.rand(200 * H, device="cuda")
    kept = src.evict_into(dst, 0, score)
    for h in range(H):
        want = ref.kept_slots(f64(src.score_view(score, 0, h)[:P]), K, 0, 0)
        assert kept.view(H, K)[h].tolist() == want
        rows = torch.tensor(want, device="cuda")
        assert torch.equal(dst.cache_view(0, "v", 0, h)[:K], src.cache_view(0, "v", 0, h)[rows])
    # a range that overlaps the source's is refused
    over = pool.state((K,), (big + P - 10,))
    with pytest.raises(rswa.RswaError) as e:
        src.evict_into(over, 0, score)
    assert e.value.status == rswa.RSWA_EINVAL


def test_evict_refusals():
    rswa = _rswa()
    src = rswa.State(1, 1, 2, 128, 4, (50,), dtype=BF, n_generated=(3,))
    score = src.score_buffer()

    def refused(dst, *args, status=None, s=src, **kw):
        with pytest.raises(rswa.RswaError) as e:
            s.evict_into(dst, *args, **kw)
        assert e.value.status == (rswa.RSWA_EINVAL if status is None else status)

    def make(**kw):
        a = dict(batch=1, num_layers=1, num_heads=2, head_dim=128, window=4, prefill_lens=(20,),
                 dtype=BF)
        a.update(kw)
        return rswa.State(**a)

    ok = make()
    refused(ok, 1, score)
    refused(ok, -1, score)
    refused(ok, 0, score, -1, 0)
    refused(ok, 0, score, 10, 11)
    refused(ok, 0, score[:-2])
    refused(ok, 0, score.double())
    refused(src, 0, score)
    refused(make(prefill_lens=(51,)), 0, score)
    for kw in (dict(num_heads=1), dict(head_dim=64), dict(window=5), dict(dtype=F32),
               dict(num_layers=2), dict(batch=2, prefill_lens=(20, 20))):
        refused(make(**kw), 0, score)
    swa = make()
    swa.set_attention(rswa.RSWA_ATTN_STANDARD_SWA)
    refused(swa, 0, score)
    empty = make(prefill_lens=(50,))
    refused(ok, 0, score, s=empty, status=rswa.RSWA_ESTATE)
    with pytest.raises(rswa.RswaError) as e:  # dst was never filled either
        ok.decode_step(0, *(torch.zeros(1, 2, 128, dtype=BF, device="cuda") for _ in range(4)))
    assert e.value.status == rswa.RSWA_ESTATE
    q = torch.zeros(1, 2, 128, dtype=BF, device="cuda")
    a, b = src.score_buffer(), src.score_buffer()
    for bad in ((a, b, a), (a, b, b), (a[:-1], b, a.clone()), (a, b.double(), a.clone())):
        with pytest.raises(rswa.RswaError):
            src.decode_step_scored(0, q, q, q, q.clone(), *bad)


@pytest.mark.parametrize("dtype,d", KINDS)
@pytest.mark.parametrize("rope", [0, 1, 2])
def test_a_state_that_took_an_eviction_serves_another_prompt(dtype, d, rope):
    """Prefilled again, it gives bit for bit what a new state gives: positions and counters are
    its own again.  A layer not prefilled yet is refused, and a later eviction counts from the
    uncut prompt as the first one did."""
    rswa = _rswa()
    H, W, P, K, L, t = 2, 6, 70, 30, 2, 9
    g = torch.Generator(device="cuda").manual_seed(rope)

    def draw(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)

    src = rswa.State(1, L, H, d, W, (P,), dtype=dtype, n_generated=(t,))
    _fill_random(src, dtype, L, 10)
    used, new = (rswa.State(1, L, H, d, W, (K,), dtype=dtype) for _ in range(2))
    for st in (src, used, new):
        if rope:
            st.set_rope(rope)
    score = torch.rand(H * (P + W), generator=g, device="cuda")

    def evict_and_step():
        out = []
        for layer in range(L):
            src.evict_into(used, layer, score)
            o = torch.empty_like(first[layer][0])
            used.decode_step(layer, *first[layer], o)
            out.append(o)
        return out

    first = [[draw(1, H, d) for _ in range(3)] for _ in range(L)]
    before = evict_and_step()
    used.advance()
    qkv = [[draw(K, H, d) for _ in range(3)] for _ in range(L)]
    outs = [[torch.empty_like(qkv[0][0]) for _ in range(L)] for _ in range(2)]
    used.prefill(0, *qkv[0], outs[0][0])
    assert used.ring()[0] == [t + 1]  # a prefill leaves the counters alone
    with pytest.raises(rswa.RswaError) as e:
        used.decode_step(1, *first[1], torch.empty_like(first[1][0]))
    assert e.value.status == rswa.RSWA_ESTATE
    used.prefill(1, *qkv[1], outs[0][1])
    used.reset_ring()
    for layer in range(L):
        new.prefill(layer, *qkv[layer], outs[1][layer])
    assert used.ring()[0] == [0]
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    tree_ins = [draw(1, 4, H, d) for _ in range(3)]
    for step in range(W + 2):
        for layer in range(L):
            x = [draw(1, H, d) for _ in range(3)]
            o = [torch.empty_like(x[0]) for _ in range(2)]
            for st, out in zip((used, new), o):
                st.decode_step(layer, *x, out)
            assert torch.equal(*o)
        o = [torch.empty_like(tree_ins[0]) for _ in range(2)]
        for st, out in zip((used, new), o):
            tree = st.tree(4)
            tree.set()
            tree.attention(0, *tree_ins, out)
            st.advance()
        assert torch.equal(*o)
    for x, y in zip(used.k_cache + used.v_cache, new.k_cache + new.v_cache):
        assert torch.equal(_bits(x), _bits(y))
    used.set_attention(rswa.RSWA_ATTN_STANDARD_SWA)  # slots are positions again
    used.set_attention(rswa.RSWA_ATTN_RING)
    for a, b in zip(before, evict_and_step()):
        assert torch.equal(a, b)
    assert used.ring()[0] == [t]
    assert used.check() == 0


def test_captured_evictions_and_prefills_in_turn():
    """A replay fills the state without a call that the host could note: every prefill after it
    still starts over, called eagerly or replayed itself, and the standard window stays refused."""
    rswa = _rswa()
    H, W, d, P, K, t = 2, 5, 128, 90, 30, 11
    src = rswa.State(1, 1, H, d, W, (P,), dtype=BF, n_generated=(t,))
    src.set_rope(rswa.RSWA_ROPE_ABSOLUTE)
    _fill_random(src, BF, 1, 13)
    dst, new = (rswa.State(1, 1, H, d, W, (K,), dtype=BF) for _ in range(2))
    new.set_rope(rswa.RSWA_ROPE_ABSOLUTE)
    g = torch.Generator(device="cuda").manual_seed(5)
    score = torch.rand(H * (P + W), generator=g, device="cuda")
    kept = torch.empty(H * K, dtype=torch.int32, device="cuda")
    qkv = [torch.randn(K, H, d, generator=g, device="cuda").to(BF) for _ in range(3)]
    x = [torch.randn(1, H, d, generator=g, device="cuda").to(BF) for _ in range(3)]
    out, pre = torch.empty_like(x[0]), torch.empty_like(qkv[0])
    new.prefill(0, *qkv, torch.empty_like(pre))
    want = torch.empty_like(out)
    new.decode_step(0, *x, want)
    src.evict_into(dst, 0, score, kept=kept)  # warm-up
    dst.prefill(0, *qkv, pre)
    torch.cuda.synchronize()
    evict, fill = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(evict):
        src.evict_into(dst, 0, score, kept=kept)
    with torch.cuda.graph(fill):
        dst.prefill(0, *qkv, pre)

    def fresh():
        dst.reset_ring()
        assert dst.ring()[0] == [0]
        out.fill_(7.0)
        dst.decode_step(0, *x, out)
        assert torch.equal(out, want)

    for again in range(3):
        evict.replay()
        assert dst.ring()[0] == [t]
        dst.prefill(0, *qkv, pre)
        fresh()
        evict.replay()
        assert dst.ring()[0] == [t]
        fill.replay()
        fresh()
        with pytest.raises(rswa.RswaError) as e:
            dst.set_attention(rswa.RSWA_ATTN_STANDARD_SWA)
        assert e.value.status == rswa.RSWA_EINVAL
    assert dst.check() == 0


def test_standard_window_is_refused_after_an_eviction():
    """The window goes by position and the kept entries' slots are not positions: the switch is
    refused, changes nothing, and the ring mode may be set again."""
    rswa = _rswa()
    H, W, d, P, K, t = 2, 30, 128, 200, 50, 3
    src = rswa.State(1, 1, H, d, W, (P,), dtype=BF, n_generated=(t,))
    dst = rswa.State(1, 1, H, d, W, (K,), dtype=BF)
    _fill_random(src, BF, 1, 9)
    dst.set_attention(rswa.RSWA_ATTN_STANDARD_SWA)  # nothing in it yet
    dst.set_attention(rswa.RSWA_ATTN_RING)
    src.evict_into(dst, 0, torch.rand(H * (P + W), device="cuda"))
    q, kn, vn = (torch.randn(1, H, d, device="cuda").to(BF) for _ in range(3))
    outs = [torch.empty_like(q) for _ in range(3)]
    dst.decode_step(0, q, kn, vn, outs[0])
    with pytest.raises(rswa.RswaError) as e:
        dst.set_attention(rswa.RSWA_ATTN_STANDARD_SWA)
    assert e.value.status == rswa.RSWA_EINVAL
    dst.decode_step(0, q, kn, vn, outs[1])
    dst.set_attention(rswa.RSWA_ATTN_RING)
    dst.decode_step(0, q, kn, vn, outs[2])
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    for h in range(H):
        held = K + t + 1
        o, mass = ref.attend(q[0, h].cpu(), dst.cache_view(0, "k", 0, h)[:held].double().cpu(),
                             dst.cache_view(0, "v", 0, h)[:held].double().cpu(), d ** -0.5)
        assert bool(((outs[0][0, h].double().cpu() - o).abs() <= ref.tolerance(o, mass, BF)).all())
    # the source keeps its whole prompt, and the choice
    src.set_attention(rswa.RSWA_ATTN_STANDARD_SWA)


def test_scored_step_and_evict_in_a_graph():
    rswa = _rswa()
    H, W, d, P, K = 2, 5, 128, 300, 100
    src = rswa.State(1, 1, H, d, W, (P,), dtype=BF, n_generated=(0,))
    dst = rswa.State(1, 1, H, d, W, (K,), dtype=BF)
    _fill_random(src, BF, 1, 5)
    q, kn, vn = (torch.randn(1, H, d, device="cuda").to(BF) for _ in range(3))
    out, out2 = torch.empty_like(q), torch.empty_like(q)
    score, scratch = src.score_buffer(), src.score_buffer()
    score2 = dst.score_buffer()
    kept = torch.empty(H * K, dtype=torch.int32, device="cuda")

    def work():
        src.decode_step_scored(0, q, kn, vn, out, score, score, scratch)
        src.advance()
        src.evict_into(dst, 0, score, 1, 1, score2, kept)
        dst.decode_step(0, q, kn, vn, out2)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work()
    for step in range(7):
        q.copy_(torch.randn(1, H, d, device="cuda"))
        kn.copy_(torch.randn(1, H, d, device="cuda"))
        graph.replay()
        assert src.ring()[0] == [step + 2] == dst.ring()[0]
        for h in range(H):
            want = ref.kept_slots(f64(src.score_view(score, 0, h)[:P]), K, 1, 1)
            assert kept.view(H, K)[h].tolist() == want
            # the decode after it ran over the kept prompt and the moved ring
            view = dst.cache_view(0, "k", 0, h)
            held = K + min(step + 3, W)
            o, mass = ref.attend(q[0, h].cpu(), view[:held].double().cpu(),
                                 dst.cache_view(0, "v", 0, h)[:held].double().cpu(), d ** -0.5)
            assert bool(((out2[0, h].double().cpu() - o).abs() <= ref.tolerance(o, mass, BF)).all())


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
def test_serve_score_evict_verify(dtype, d):
    """The operators as a server would use them: prefill, scored decode steps over two layers,
    eviction to a smaller state, then drafted trees verified and committed over it, every
    attention output against the 64-bit definition over the entries that are left."""
    rswa = _rswa()
    L, H, W, plens, keep, T, steps = 2, 2, 6, (400, 90), (130, 90), 7, 8
    B = len(plens)
    ms = [ref.Model(plens, W, H, d, dtype, seed=30 + x) for x in range(L)]
    st = rswa.State(B, L, H, d, W, plens, dtype=dtype)
    for layer, m in enumerate(ms):
        q = m.draw(sum(plens), H, d).cuda()
        st.prefill(layer, q, torch.cat(m.pk).cuda(), torch.cat(m.pv).cuda(), torch.empty_like(q))
    scores, scratch = [st.score_buffer() for _ in range(L)], st.score_buffer()
    for _ in range(steps):
        for layer, m in enumerate(ms):
            q, kn, vn = (m.draw(B, H, d) for _ in range(3))
            out = torch.empty(B, H, d, dtype=dtype, device="cuda")
            st.decode_step_scored(layer, q.cuda(), kn.cuda(), vn.cuda(), out, scores[layer],
                                  scores[layer], scratch)
            for b in range(B):
                m.gk[b].append(kn[b])
                m.gv[b].append(vn[b])
        st.advance()
    small = rswa.State(B, L, H, d, W, keep, dtype=dtype)
    left = []
    for layer, m in enumerate(ms):
        kept = st.evict_into(small, layer, scores[layer], 2, 3).cpu()
        base, rows = 0, {}
        for b in range(B):
            for h in range(H):
                rows[b, h] = kept[base:base + keep[b]].long()
                base += keep[b]
        left.append(rows)
    st.close()
    tree = small.tree(T)
    rng = np.random.default_rng(1)
    for _ in range(4):
        parents = [ref.random_parents(rng, T) for _ in range(B)]
        paths = [ref.path_of(p, int(rng.integers(0, T))) for p in parents]
        tree.set(_ints(parents))
        ks, vs = [], []
        for layer, m in enumerate(ms):
            q, k, v = (m.draw(B, T, H, d) for _ in range(3))
            out = torch.empty(B, T, H, d, dtype=dtype, device="cuda")
            tree.attention(layer, q.cuda(), k.cuda(), v.cuda(), out)
            out = out.cpu()
            for b in range(B):
                for i in range(T):
                    p = ref.path_of(parents[b], i)
                    for h in range(H):
                        kk, vv = m.entries(b, h, [k[b, x] for x in p], [v[b, x] for x in p])
                        r = left[layer][b, h]
                        kk = torch.cat([kk[:plens[b]][r], kk[plens[b]:]])
                        vv = torch.cat([vv[:plens[b]][r], vv[plens[b]:]])
                        o, mass = ref.attend(q[b, i, h], kk, vv, d ** -0.5)
                        err = (out[b, i, h].double() - o).abs()
                        assert bool((err <= ref.tolerance(o, mass, dtype)).all())
            ks.append(k.cuda())
            vs.append(v.cuda())
            for b, p in enumerate(paths):
                m.gk[b] += [k[b, x] for x in p]
                m.gv[b] += [v[b, x] for x in p]
        tree.commit(ks, vs, _ints([p + [0] * (T - len(p)) for p in paths]),
                    _ints([len(p) for p in paths]))
        tree.advance()
        assert small.ring()[0] == [len(x) for x in ms[0].gk]
    assert small.check() == 0
