"""Measured cases of the draft-tree and cache-eviction operators.

Four operators over the ring cache (a prompt of P_b tokens plus a ring of the W
most recently generated ones, head-major rows, one K and one V buffer a layer):

  tree    attention of a tree of drafted tokens over the cache, all layers of a
          verification pass (the tree's masks are set once, then one call a layer);
  commit  the accepted path's keys and values into the ring slots of every layer;
  scored  a decode step that also accumulates every cache entry's softmax weight;
  evict   the prompt entries with the highest accumulated weight moved, with the
          ring, into a smaller cache.

`own` chooses between the library's calls and the plain form of the same
definitions in elementary torch operations.
"""
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _case(name, op, dtype, batch, layers, heads, dim, window, p_lo, p_hi, t_lo, t_hi, **more):
    return {"name": name, "op": op, "dtype": dtype, "batch": batch, "layers": layers,
            "heads": heads, "dim": dim, "window": window, "p_lo": p_lo, "p_hi": p_hi,
            "t_lo": t_lo, "t_hi": t_hi, "lens_seed": more.pop("lens_seed", 5), **more}


def listed():
    return [
        # one page (4 views x 256 image tokens + 64 text), a few drafted tokens, all
        # 12 layers: the latency of one verification pass for one user
        _case("tree_page_8", "tree", "bf16", 1, 12, 10, 128, 128, 1088, 1088, 500, 500,
              draft=8, draft_lo=8, chain=False),
        # 32-page documents, 8 users, a middling tree
        _case("tree_pages_32", "tree", "bf16", 8, 2, 10, 128, 128, 8256, 8256, 300, 300,
              draft=32, draft_lo=32, chain=False),
        # near the position limit, a wide tree: the largest read of the cache
        _case("tree_long_64", "tree", "bf16", 4, 1, 10, 128, 128, 32640, 32640, 1000, 1000,
              draft=64, draft_lo=64, chain=False),
        # a serving batch: ragged prompts, rings in every state of filling, odd and
        # ragged draft counts
        _case("tree_ragged_17", "tree", "bf16", 64, 1, 10, 128, 128, 1024, 16384, 0, 128,
              draft=17, draft_lo=1, chain=False),
        # single precision and the small head, drafted as a chain
        _case("tree_fp32_16", "tree", "fp32", 2, 2, 10, 64, 100, 1088, 1088, 37, 37,
              draft=16, draft_lo=16, chain=True),
        # the accepted tokens of one user into 12 layers: launch latency
        _case("commit_page", "commit", "bf16", 1, 12, 10, 128, 128, 1088, 1088, 500, 500,
              draft=8, draft_lo=3),
        # a serving batch's accepted tokens; some sequences accept none
        _case("commit_serving", "commit", "bf16", 64, 12, 10, 128, 128, 64, 300, 0, 400,
              draft=32, draft_lo=0),
        # one page, all layers, weights accumulated at every step
        _case("scored_page", "scored", "bf16", 1, 12, 10, 128, 128, 1088, 1088, 500, 500),
        # near the position limit: the largest read of the cache
        _case("scored_long", "scored", "bf16", 4, 1, 10, 128, 128, 32640, 32640, 1000, 1000),
        # single precision, small head, one page kept at a third
        _case("evict_page_fp32", "evict", "fp32", 1, 2, 10, 64, 128, 1088, 1088, 500, 500,
              keep=0.34, first=4, last=64),
        # 32-page documents cut to half
        _case("evict_pages", "evict", "bf16", 8, 1, 10, 128, 128, 8256, 8256, 300, 300,
              keep=0.5, first=64, last=256),
        # the longest prompts cut to a quarter
        _case("evict_long", "evict", "bf16", 4, 1, 10, 128, 128, 32640, 32640, 1000, 1000,
              keep=0.25, first=64, last=256),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread evenly over its logarithm."""
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(["tree", "tree", "commit", "scored", "evict"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    heads, dim = rng.choice([2, 5, 8, 10, 16]), rng.choice([64, 128, 128])
    layers = rng.choice([1, 2, 3])
    window = rng.choice([128, 128, _log(rng, 128, 500)])
    batch = _log(rng, 1, 64)
    draft = _log(rng, 1, 128) if op in ("tree", "commit") else 1
    if op == "commit":
        p_hi = _log(rng, 16, 400)
    else:
        # bounded by the largest listed read of the cache and its products
        room = 4 * 32640 * 10 // (batch * heads * layers)
        if op == "tree":
            room = min(room, 4 * 32640 * 10 * 64 // (batch * heads * layers * draft))
        if dtype == "fp32":
            room //= 4
        p_hi = _log(rng, 32, max(33, min(32640, room)))
    p_lo = p_hi if rng.random() < 0.5 else max(1, p_hi // 8)
    t_hi = rng.choice([window, 5, 3 * window])
    more = {"lens_seed": rng.randrange(1 << 20)}
    if op in ("tree", "commit"):
        more.update(draft=draft, draft_lo=rng.choice([draft, 0]))
    if op == "tree":
        more.update(chain=rng.random() < 0.25)
    if op == "evict":
        more.update(keep=round(0.1 + 0.8 * rng.random(), 2), first=rng.choice([0, 1, 3]),
                    last=rng.choice([0, 1]))
    case = _case("", op, dtype, batch, layers, heads, dim, window, p_lo, p_hi,
                 rng.choice([0, t_hi]), t_hi, **more)
    del case["name"]
    return case


def _lens(case):
    """Host values of a case: prompt lengths, tokens generated, drafted or accepted tokens."""
    r = random.Random(case["lens_seed"])
    B = case["batch"]
    plen = [r.randint(case["p_lo"], case["p_hi"]) for _ in range(B)]
    t = [r.randint(case["t_lo"], case["t_hi"]) for _ in range(B)]
    n = [r.randint(case.get("draft_lo", 0), case.get("draft", 0)) for _ in range(B)]
    return plen, t, n


def _kept(case, plen):
    return [min(p, max(case["first"] + case["last"], int(p * case["keep"]))) for p in plen]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = random.Random(seed)
    dt, op = DTYPES[case["dtype"]], case["op"]
    B, L, H, d, W = (case[x] for x in ("batch", "layers", "heads", "dim", "window"))
    plen, t, n = _lens(case)
    rows = H * sum(p + W for p in plen)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dt)

    def ints(x, kind=torch.int32):
        return torch.tensor(x, dtype=kind, device="cuda")

    st = {"case": case, "plen": plen, "rows": rows, "t": ints(t, torch.int64),
          "plen_dev": ints(plen, torch.int64), "scale": d ** -0.5}
    slots = [p + W for p in plen]
    st["base_dev"] = ints([H * sum(slots[:b]) for b in range(B)], torch.int64)
    st["len_dev"] = ints(slots, torch.int64)
    st["k"] = [normal(rows, d) for _ in range(L)]
    st["v"] = [normal(rows, d) for _ in range(L)]
    if op in ("tree", "commit"):
        T = case["draft"]
        st["n"] = ints(n)
        st["kd"] = [normal(B, T, H, d) for _ in range(L)]
        st["vd"] = [normal(B, T, H, d) for _ in range(L)]
        parent = [[i - 1 if case.get("chain") else r.randint(max(-1, i - 6), i - 1)
                   for i in range(T)] for _ in range(B)]
        if op == "tree":
            st["q"] = [normal(B, T, H, d) for _ in range(L)]
            st["out"] = [torch.zeros(B, T, H, d, device="cuda", dtype=dt) for _ in range(L)]
        else:
            # the accepted path: a chain down from a first node, of n tokens
            path = [[0] * T for _ in range(B)]
            for b in range(B):
                nodes = sorted(r.sample(range(T), n[b]))
                for i, x in enumerate(nodes):
                    path[b][i] = x
                    parent[b][x] = nodes[i - 1] if i else -1
            st["path"] = ints(path)
        st["parent"] = ints(parent)
    if op == "scored":
        st["q"], st["kn"], st["vn"] = ([normal(B, H, d) for _ in range(L)] for _ in range(3))
        st["out"] = [torch.empty(B, H, d, device="cuda", dtype=dt) for _ in range(L)]
        st["score_in"] = [torch.rand(rows, generator=g, device="cuda") for _ in range(L)]
        st["score_out"] = [torch.zeros(rows, device="cuda") for _ in range(L)]
        st["scratch"] = torch.empty(rows, device="cuda")
    if op == "evict":
        keep = _kept(case, plen)
        st["keep"] = keep
        drows = H * sum(p + W for p in keep)
        # accumulated weights: many small, a few large, a share of exact ties at zero
        st["score"] = [torch.rand(rows, generator=g, device="cuda").pow(8) *
                       (torch.rand(rows, generator=g, device="cuda") > 0.3) for _ in range(L)]
        st["k2"] = [torch.zeros(drows, d, device="cuda", dtype=dt) for _ in range(L)]
        st["v2"] = [torch.zeros(drows, d, device="cuda", dtype=dt) for _ in range(L)]
        st["score2"] = [torch.zeros(drows, device="cuda") for _ in range(L)]
        st["kept"] = [torch.empty(H * sum(keep), device="cuda", dtype=torch.int32)
                      for _ in range(L)]
        st["kept_base"] = ints([H * sum(keep[:b]) for b in range(B)], torch.int64)
        st["base2_dev"] = ints([H * sum(p + W for p in keep[:b]) for b in range(B)], torch.int64)
        st["keep_dev"] = ints(keep, torch.int64)
    if own:
        from ring_sliding_window_b200 import rswa

        def state(lens, k, v):
            s = rswa.State(B, L, H, d, W, lens, dtype=dt, n_generated=t)
            for layer in range(L):
                k[layer] = s.k_cache[layer].view(-1, d).copy_(k[layer])
                v[layer] = s.v_cache[layer].view(-1, d).copy_(v[layer])
            return s

        st["state"] = state(plen, st["k"], st["v"])
        if op in ("tree", "commit"):
            st["tree"] = st["state"].tree(case["draft"])
        if op == "commit":
            st["tree"].set(st["parent"])
        if op == "evict":
            st["state2"] = state(st["keep"], st["k2"], st["v2"])
    return st


def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state)


# ------------------------------------------------------------ the library's calls
def _own_tree(st):
    st["tree"].set(st["parent"], st["n"])
    for layer, out in enumerate(st["out"]):
        st["tree"].attention(layer, st["q"][layer], st["kd"][layer], st["vd"][layer], out)
    return st["out"]


def _own_commit(st):
    st["tree"].commit(st["kd"], st["vd"], st["path"], st["n"])
    return st["k"], st["v"]


def _own_scored(st):
    for layer, out in enumerate(st["out"]):
        st["state"].decode_step_scored(layer, st["q"][layer], st["kn"][layer], st["vn"][layer], out,
                                       st["score_in"][layer], st["score_out"][layer],
                                       st["scratch"])
    return st["out"], st["score_out"], st["k"], st["v"]


def _own_evict(st):
    case = st["case"]
    for layer, kept in enumerate(st["kept"]):
        st["state"].evict_into(st["state2"], layer, st["score"][layer], case["first"], case["last"],
                               st["score2"][layer], kept)
    return st["k2"], st["v2"], st["score2"], st["kept"]


# ------------------------------------------------------------------ plain forms
def _index(st):
    """Cache rows of every (sequence, head, slot), the longest sequence's slots for all:
    [B, H, Lmax] row numbers (clamped where a sequence is shorter) and [B, Lmax] slots."""
    H, Lmax = st["case"]["heads"], max(st["plen"]) + st["case"]["window"]
    s = torch.arange(Lmax, device="cuda")
    h = torch.arange(H, device="cuda")
    slot = torch.minimum(s, st["len_dev"][:, None] - 1)
    rows = st["base_dev"][:, None, None] + h[:, None] * st["len_dev"][:, None, None] + slot[:, None]
    return rows, s.expand(len(st["plen"]), Lmax)


def _entries(st, buf, rows):
    """The cache's entries as [B, H, Lmax, d] in 32 bits."""
    case = st["case"]
    if case["p_lo"] == case["p_hi"]:
        return buf.view(case["batch"], case["heads"], -1, case["dim"]).float()
    return buf[rows].float()


def _ages(st, slot):
    """Tokens since each ring entry was generated (0 for the prompt), and whether a slot
    holds an entry at all; [B, Lmax]."""
    W, t = st["case"]["window"], st["t"][:, None]
    r = slot - st["plen_dev"][:, None]
    age = torch.where(r < 0, 0, (t - 1 - r) % W + 1)
    held = (r < 0) | ((r < W) & (r < t))
    return age, held


def _ancestors(parent):
    """[B, T, T] truth values (node i has node j above it, or is it) and depths [B, T]."""
    B, T = parent.shape
    up = torch.nn.functional.one_hot(parent.long() + 1, T + 1)[:, :, 1:].float()
    seen = torch.eye(T, device="cuda").expand(B, T, T)
    reach, step = seen + up, up
    for _ in range(T.bit_length()):  # paths of up to 2, 4, 8, ... steps
        step = step @ step
        reach = ((reach + step @ reach) > 0).float()
    return reach > 0, reach.sum(-1).long() - 1


def _plain_tree(st):
    W, T = st["case"]["window"], st["case"]["draft"]
    rows, slot = _index(st)
    age, held = _ages(st, slot)
    above, depth = _ancestors(st["parent"])
    real = torch.arange(T, device="cuda") < st["n"][:, None]
    far = age[:, None] + depth[:, :, None] > W - 1
    see_cache = held[:, None] & ((age == 0)[:, None] | ~far)               # [B, T, Lmax]
    see_draft = above & (depth[:, None] >= depth[:, :, None] - W + 1)      # [B, T, T]
    see = torch.cat([see_cache, see_draft], -1)[:, None]
    for layer, out in enumerate(st["out"]):
        q = st["q"][layer].float().transpose(1, 2)
        k = torch.cat([_entries(st, st["k"][layer], rows),
                       st["kd"][layer].float().transpose(1, 2)], 2)
        s = (q @ k.transpose(2, 3) * st["scale"]).masked_fill(~see, float("-inf"))
        p = torch.exp(s - s.amax(-1, keepdim=True))
        del s, k
        v = torch.cat([_entries(st, st["v"][layer], rows),
                       st["vd"][layer].float().transpose(1, 2)], 2)
        o = (p @ v / p.sum(-1, keepdim=True)).transpose(1, 2).to(out.dtype)
        out.copy_(torch.where(real[:, :, None, None], o, out))
    return st["out"]


def _plain_commit(st):
    case = st["case"]
    W, T, H = case["window"], case["draft"], case["heads"]
    i = torch.arange(T, device="cuda")
    slot = st["plen_dev"][:, None] + (st["t"][:, None] + i) % W           # [B, T]
    h = torch.arange(H, device="cuda")
    rows = (st["base_dev"][:, None, None] + h * st["len_dev"][:, None, None] + slot[:, :, None])
    real = (i < st["n"][:, None])[:, :, None, None]
    pick = st["path"].long()[:, :, None, None].expand(-1, -1, H, case["dim"])
    for cache, drafted in zip(st["k"] + st["v"], st["kd"] + st["vd"]):
        cache[rows] = torch.where(real, drafted.gather(1, pick), cache[rows])
    return st["k"], st["v"]


def _plain_scored(st):
    case = st["case"]
    W = case["window"]
    rows, slot = _index(st)
    h = torch.arange(case["heads"], device="cuda")
    new = st["plen_dev"] + st["t"] % W
    new_rows = st["base_dev"][:, None] + h * st["len_dev"][:, None] + new[:, None]   # [B, H]
    held = slot < (st["plen_dev"] + torch.minimum(st["t"] + 1, torch.tensor(W)))[:, None]
    fresh = (slot == new[:, None])[:, None]
    inside = held[:, None].expand(-1, case["heads"], -1)
    for layer, out in enumerate(st["out"]):
        st["k"][layer][new_rows] = st["kn"][layer]
        st["v"][layer][new_rows] = st["vn"][layer]
        k = _entries(st, st["k"][layer], rows)
        s = (k @ st["q"][layer].float()[..., None])[..., 0] * st["scale"]
        s = s.masked_fill(~held[:, None], float("-inf"))
        p = torch.exp(s - s.amax(-1, keepdim=True))
        p = p / p.sum(-1, keepdim=True)
        out.copy_((p[:, :, None] @ _entries(st, st["v"][layer], rows))[:, :, 0])
        total = p + st["score_in"][layer][rows].masked_fill(fresh, 0.0)
        st["score_out"][layer][rows[inside]] = total[inside]
    return st["out"], st["score_out"], st["k"], st["v"]


def _plain_evict(st):
    case = st["case"]
    H, W = case["heads"], case["window"]
    rows, slot = _index(st)
    P, K = st["plen_dev"][:, None], st["keep_dev"][:, None]
    guarded = (slot < case["first"]) | (slot >= P - case["last"])
    j = torch.arange(max(st["keep"]) + W, device="cuda")
    h = torch.arange(H, device="cuda")
    # destination slot j: a kept prompt entry while j < K, then ring slot j - K if held
    is_kept = (j < K)[:, None].expand(-1, H, -1)
    full = torch.minimum(st["t"], torch.tensor(W))[:, None]
    valid = (is_kept | (j < K + full)[:, None])
    to = st["base2_dev"][:, None, None] + h[:, None] * (K + W)[:, None] + j
    kept_at = (st["kept_base"][:, None, None] + h[:, None] * K[:, None] + j)[is_kept]
    for layer, kept in enumerate(st["kept"]):
        rank = st["score"][layer][rows].masked_fill(guarded[:, None], float("inf"))
        rank = rank.masked_fill((slot >= P)[:, None], float("-inf"))
        order = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :j.numel()]
        order = torch.where(is_kept, order, 1 << 40)
        order = torch.sort(order, dim=-1).values
        src = torch.where(is_kept, order, (P + j - K)[:, None])
        kept[kept_at] = src[is_kept].int()
        at = st["base_dev"][:, None, None] + h[:, None] * st["len_dev"][:, None, None] + src
        at, dst = at[valid], to[valid]
        st["k2"][layer][dst] = st["k"][layer][at]
        st["v2"][layer][dst] = st["v"][layer][at]
        st["score2"][layer][dst] = st["score"][layer][at]
    return st["k2"], st["v2"], st["score2"], st["kept"]


_plain = {"tree": _plain_tree, "commit": _plain_commit, "scored": _plain_scored,
          "evict": _plain_evict}
_own = {"tree": _own_tree, "commit": _own_commit, "scored": _own_scored, "evict": _own_evict}


# --------------------------------------------------------------- work and truth
def work(case):
    """Each input read once, each output written once; two operations a product."""
    plen, t, n = _lens(case)
    L, H, d, W = (case[x] for x in ("layers", "heads", "dim", "window"))
    es = 2 if case["dtype"] == "bf16" else 4
    row = 2 * H * d * es  # a token's K and V
    if case["op"] == "tree":
        keys = [p + min(x, W) for p, x in zip(plen, t)]
        byte = L * sum(k * row + x * 2 * row for k, x in zip(keys, n)) + 8 * len(n) * case["draft"]
        return {"bytes": byte, "flops": L * sum(4 * x * H * d * (k + (x + 1) // 2)
                                                for k, x in zip(keys, n))}
    if case["op"] == "commit":
        return {"bytes": L * 2 * row * sum(n) + 4 * case["draft"] * len(n), "flops": 0}
    if case["op"] == "scored":
        keys = [p + min(x + 1, W) for p, x in zip(plen, t)]
        return {"bytes": L * sum(k * (row + 8 * H) + 3 * row for k in keys),
                "flops": L * sum(4 * H * d * k for k in keys)}
    keep = _kept(case, plen)
    moved = sum(k + min(x, W) for k, x in zip(keep, t))
    return {"bytes": L * (2 * moved * (row + 4 * H) + 4 * H * (sum(plen) + sum(keep))),
            "flops": 0}


def exact(case, seed):
    """Attention outputs and accumulated weights in 64 bits, sequence by sequence from the
    definition; entries that are only moved have no computed value."""
    if case["op"] in ("commit", "evict"):
        return None
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    H, d, W, L = case["heads"], case["dim"], case["window"], case["layers"]
    plen, t, n = _lens(case)

    def caches(layer, b):
        lo = H * sum(p + W for p in plen[:b])
        shape = (H, plen[b] + W, d)
        part = slice(lo, lo + shape[0] * shape[1])
        return st["k"][layer][part].view(shape), st["v"][layer][part].view(shape), part

    def softmax(s):
        e = torch.exp(s - s.max(-1, keepdim=True).values)
        return e / e.sum(-1, keepdim=True)

    outs, scores = [], []
    if case["op"] == "scored":
        for layer in range(L):
            o = torch.zeros(case["batch"], H, d, dtype=torch.float64, device="cuda")
            sc = torch.zeros(st["rows"], dtype=torch.float64, device="cuda")
            for b in range(case["batch"]):
                k, v, part = caches(layer, b)
                have = plen[b] + min(t[b] + 1, W)
                new = plen[b] + t[b] % W
                k, v = k[:, :have].double(), v[:, :have].double()
                k[:, new], v[:, new] = st["kn"][layer][b].double(), st["vn"][layer][b].double()
                w = softmax(torch.einsum("hd,hsd->hs", st["q"][layer][b].double(), k) * d ** -0.5)
                o[b] = torch.einsum("hs,hsd->hd", w, v)
                before = st["score_in"][layer][part].view(H, -1)[:, :have].double()
                before[:, new] = 0
                sc[part].view(H, -1)[:, :have] = before + w
            outs.append(o)
            scores.append(sc)
        return outs, scores, [None] * L, [None] * L
    parents = st["parent"].tolist()
    for layer in range(L):
        o = torch.zeros(case["batch"], case["draft"], H, d, dtype=torch.float64, device="cuda")
        for b in range(case["batch"]):
            if n[b] == 0:
                continue
            k, v, _ = caches(layer, b)
            have = plen[b] + min(t[b], W)
            k = torch.cat([k[:, :have], st["kd"][layer][b, :n[b]].transpose(0, 1)], 1).double()
            v = torch.cat([v[:, :have], st["vd"][layer][b, :n[b]].transpose(0, 1)], 1).double()
            # the generated token number that each entry holds; the prompt is always seen
            number = {plen[b] + x % W: x for x in range(max(0, t[b] - W), t[b])}
            seen = torch.zeros(n[b], have + n[b], dtype=torch.bool)
            for i in range(n[b]):
                chain = [i]
                while parents[b][chain[-1]] >= 0:
                    chain.append(parents[b][chain[-1]])
                oldest = t[b] + len(chain) - 1 - W + 1
                seen[i, :plen[b]] = True
                for s, x in number.items():
                    seen[i, s] = x >= oldest
                for up, node in enumerate(chain):
                    seen[i, have + node] = up < W
            s = torch.einsum("thd,hsd->hts", st["q"][layer][b, :n[b]].double(), k) * d ** -0.5
            w = softmax(s.masked_fill(~seen.to(s.device), float("-inf")))
            o[b, :n[b]] = torch.einsum("hts,hsd->thd", w, v)
        outs.append(o)
    return outs
