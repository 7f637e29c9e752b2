"""OwnerShard and OwnerShard8 as objects: what they are made from, saved to and refuse.  On the CPU:
layouts, tables and checkpoints only, nothing is launched."""
import copy

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import zero_sharded_optimizer_owned_amd as zs  # noqa: E402

CLASSES = [zs.OwnerShard, zs.OwnerShard8]


@pytest.mark.parametrize("cls", CLASSES)
def test_sizes_from_any_iterable(cls):
    want = cls([1000, 37, 5003], 4, 1, device="cpu")
    model = [torch.zeros(1000), torch.zeros(37), torch.zeros(5003)]
    for numels in ((p.numel() for p in model), map(len, model), {k: len(p) for k, p in enumerate(model)}.values(),
                   (1000, 37, 5003), torch.Size([1000, 37, 5003]), np.array([1000, 37, 5003]),
                   np.array([1000, 37, 5003], dtype=np.uint64), [torch.tensor(1000), np.int32(37), 5003]):
        got = cls(numels, 4, 1, device="cpu")
        assert got.numels == want.numels == [1000, 37, 5003] and all(type(n) is int for n in got.numels)
        assert (got.begin, got.end, got.local_base) == (want.begin, want.end, want.local_base)
        assert np.array_equal(got.chunks, want.chunks) and np.array_equal(got.dense_offsets, want.dense_offsets)


@pytest.mark.parametrize("cls", CLASSES)
@pytest.mark.parametrize("numels, error", [([-5], OverflowError), (np.array([3, -5]), OverflowError), (5, TypeError),
                                           ([[1, 2], [3, 4]], TypeError), ([4, 0], zs.ZeroShardError)])
def test_sizes_that_are_none(cls, numels, error):
    with pytest.raises(error):
        cls(numels, 1, 0, device="cpu")


@pytest.mark.parametrize("cls, other", [CLASSES, CLASSES[::-1]])
def test_a_checkpoint_of_the_other_width_is_refused_whole(cls, other, tmp_path):
    """Nothing of the owner changes when its load is refused."""
    saved, mine = other([300, 7], 2, 1, device="cpu"), cls([300, 7], 2, 1, device="cpu")
    saved.alloc_state()
    saved.master.fill_(7.0)
    saved.save(str(tmp_path / "s.npz"), 3)
    mine.alloc_state()
    before = mine.master.clone()
    with pytest.raises(ValueError):
        mine.load(str(tmp_path / "s.npz"))
    assert torch.equal(mine.master, before)
    again = other([300, 7], 2, 1, device="cpu")
    assert again.load(str(tmp_path / "s.npz")) == 3 and torch.equal(again.master, saved.master)


@pytest.mark.parametrize("cls", CLASSES)
def test_the_constructor_makes_every_table(cls, monkeypatch):
    """An export or import later builds nothing (it may run under a graph's capture, or on several threads)."""
    sh = cls([100] * 50 + [5003], 2, 1, device="cpu")

    def no(*a, **k):
        raise AssertionError("a table made after construction")

    for name in ("zero_chunk_table", "zero_chunk_groups", "zero_dense_offsets", "zero_piece_table", "chunks_to_device"):
        monkeypatch.setattr(zs, name, no)
    assert sh.chunks.size and sh.n_groups == sh.groups.size - 1 and sh.dense_total == 10_003 and sh.n_real
    assert sh.chunks_dev.numel() == 16 * sh.chunks.size
    assert sh.tensor_offset_dev.numel() == sh.dense_offset_dev.numel() == 51


def test_device_0_is_a_device(monkeypatch):
    """Not the current one."""
    seen = []
    make = lambda *a, device, **k: seen.append(device)  # noqa: E731
    monkeypatch.setattr(torch, "zeros", make)
    monkeypatch.setattr(torch, "empty", make)
    for call in (lambda d: zs.policy_workspace(3, device=d), lambda d: zs.preference_workspace(3, 1, device=d),
                 lambda d: zs.check_workspace(3, device=d)):
        for device, want in ((0, 0), (1, 1), (None, "cuda"), ("cuda:0", "cuda:0")):
            call(device)
            assert seen.pop() == want
    monkeypatch.undo()
    monkeypatch.setattr(torch, "device", lambda d: seen.append(d) or "cpu")
    zs.OwnerShard([5], 1, 0, device=0)
    assert seen == [0]


def test_a_copy_of_an_owner_uses_its_own_tables(monkeypatch):
    """No address outlives the tensor it belongs to: a deep copy after a call, or one with a new table."""
    sh = zs.OwnerShard8([100] * 40, 2, 1, device="cpu")
    sh.alloc_state()
    monkeypatch.setattr(zs, "_device_stream", lambda: (-1, 0))  # where a host tensor's get_device() is
    tables = lambda s: s._checked()[2][0:3:2]  # noqa: E731
    own = lambda s: (s.pieces_dev.data_ptr(), s.masks_dev.data_ptr())  # noqa: E731
    assert tables(sh) == own(sh)
    twin = copy.deepcopy(sh)
    assert tables(twin) == own(twin) and not set(own(twin)) & set(own(sh))
    sh.pieces_dev = sh.pieces_dev.clone()
    assert tables(sh) == own(sh)


@pytest.mark.parametrize("change", [dict(n_pieces=-1), dict(begin=-8, end=-8), dict(end=-1)])
def test_negative_counts_are_refused(change, monkeypatch):
    """They are unsigned for the library: -1 pieces would be all there is of memory."""
    sh = zs.OwnerShard8([1000], 1, 0, device="cpu")
    sh.alloc_state()
    monkeypatch.setattr(zs, "_device_stream", lambda: (-1, 0))
    monkeypatch.setattr(zs, "_check", lambda rc: None)
    monkeypatch.setattr(zs, "lib", lambda: pytest.fail("reached the library"))
    state, moments = {**sh._state8(), **change}, [torch.zeros(1024), torch.zeros(1024)]
    hyper = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8)
    for call in (lambda: zs.zero_adam8_step(**state, master=sh.master, step=1, reduced_g=moments[0], **hyper),
                 lambda: zs.zero_moments8_pack(**state, exp_avg=moments[0], exp_avg_sq=moments[1]),
                 lambda: zs.zero_moments8_unpack(**state, exp_avg=moments[0], exp_avg_sq=moments[1])):
        with pytest.raises(ValueError):
            call()
