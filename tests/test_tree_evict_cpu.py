"""Host-side checks of the draft-tree and eviction calls: refused before anything is
launched, on any machine."""
import pytest


@pytest.fixture(scope="module")
def rswa():
    from ring_sliding_window_b200 import build
    build.build()
    from ring_sliding_window_b200 import rswa as mod
    return mod


A = 4096  # an aligned stand-in address, never dereferenced on these paths


def test_null_objects_are_refused(rswa):
    lib, E = rswa.lib, rswa.RSWA_EINVAL
    out = rswa.ctypes.c_void_p()
    assert lib.rswa_tree_workspace_bytes(None, 8) == 0
    assert lib.rswa_tree_create(None, 8, A, 1 << 20, None, rswa.ctypes.byref(out)) == E
    assert lib.rswa_tree_create(None, 8, A, 1 << 20, None, None) == E
    assert lib.rswa_tree_destroy(None) == E
    assert lib.rswa_tree_set(None, None, None, None) == E
    assert lib.rswa_tree_attention(None, 0, A, A, A, A, None) == E
    assert lib.rswa_tree_commit(None, None, None, A, A, None) == E
    assert lib.rswa_tree_advance(None, None) == E
    assert lib.rswa_score_bytes(None) == 0
    assert lib.rswa_decode_step_scored(None, 0, A, A, A, A, A, A, A, None) == E
    assert lib.rswa_evict(None, None, 0, A, 0, 0, A, A, None) == E


def test_reference_kept_slots():
    """The tests' own definition, on a hand-made case."""
    import tree_reference as ref
    nan = float("nan")
    assert ref.kept_slots([1, 3, 3, 2, nan, 0], 2, 0, 0) == [1, 2]
    assert ref.kept_slots([1, 3, 3, 2, nan, 0], 3, 1, 1) == [0, 1, 5]
    assert ref.kept_slots([0.0, -0.0, nan], 1, 0, 0) == [0]
    assert ref.kept_slots([nan, 0.0], 1, 0, 0) == [1]


def test_reference_paths():
    import tree_reference as ref
    assert ref.path_of([-1, 0, 0, 2], 3) == [0, 2, 3]
    assert ref.path_of([-1, -1], 1) == [1]


@pytest.mark.parametrize("n", [12, 300, 2000, 16000])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("positive", [False, True])
def test_the_pair_bound_needs_the_second_half_of_a_weight(n, d, positive):
    """Weights as bf16 pairs keep the bound of tree_reference.pair_tolerance; without the second
    value, with it subtracted or doubled, some of the outputs break it."""
    import torch

    import tree_reference as ref
    g = torch.Generator().manual_seed(n + d)
    broken = {0.0: 0, -1.0: 0, 2.0: 0}
    for _ in range(20 if n <= 2000 else 3):
        q, k, v = (torch.randn(*s, generator=g).to(torch.bfloat16).double()
                   for s in ((d,), (n, d), (n, d)))
        if positive:
            v = v.abs()
        o, mass = ref.attend(q, k, v, d ** -0.5)
        lim = ref.pair_tolerance(q, k, o, mass, d ** -0.5)
        assert bool(((ref.pair_attend(q, k, v, d ** -0.5) - o).abs() <= lim).all())
        for lo in broken:
            err = (ref.pair_attend(q, k, v, d ** -0.5, lo) - o).abs()
            broken[lo] += int((err > lim).sum())
    if positive or n <= 300:  # (sums that cancel hide it among many entries)
        assert all(x > 0 for x in broken.values()), broken


def test_a_tree_of_a_closed_state_is_refused(rswa, monkeypatch):
    """The C tree points to the C state: once that is gone no call may reach the library.  The
    library's calls are replaced here by ones that only note that they were made."""
    import types

    import torch

    class StandIn(rswa.Tree):
        def __del__(self):
            pass

    made = []
    for name in ("set", "attention", "commit", "advance", "destroy"):
        monkeypatch.setattr(rswa, f"rswa_tree_{name}", lambda *a, name=name: made.append(name))
    B, T, H, d = 2, 3, 2, 64
    st = types.SimpleNamespace(B=B, L=1, H=H, d=d, dtype=torch.float32, handle=1,
                               _device=torch.device("cpu"))
    tree = StandIn.__new__(StandIn)
    tree.state, tree.T, tree._shape, tree.handle = st, T, (B, T, H, d), 2
    x = [torch.zeros(B, T, H, d) for _ in range(4)]
    path, n = torch.zeros(B, T, dtype=torch.int32), torch.zeros(B, dtype=torch.int32)
    calls = [lambda: tree.set(path, n), lambda: tree.attention(0, *x),
             lambda: tree.commit(x[:1], x[1:2], path, n), lambda: tree.advance()]
    for call in calls:
        call()
    assert made == ["set", "attention", "commit", "advance"]
    made.clear()
    st.handle = None  # as State.close() leaves it
    for call in calls:
        with pytest.raises(rswa.RswaError) as e:
            call()
        assert e.value.status == rswa.RSWA_EINVAL
    assert made == []
    tree.close()  # the tree's own memory is still there to be freed
    assert made == ["destroy"]
    st.handle = 1
    for call in calls:  # a closed tree
        with pytest.raises(rswa.RswaError) as e:
            call()
        assert e.value.status == rswa.RSWA_EINVAL
    assert made == ["destroy"]
