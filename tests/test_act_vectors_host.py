"""CPU tests of what the activation checkpoints' binding does with tensors whose
memory changes between calls."""
import pytest
import torch

BF16, CPU = torch.bfloat16, torch.device("cpu")


@pytest.fixture(scope="module")
def ps():
    import precision_state_amd as ps
    return ps


def vectors(ps, **kw):
    v = dict(post_weight=torch.ones(8), gate=torch.ones(3, 8), mul=torch.ones(3, 8), add=torch.ones(3, 8),
             segments=torch.tensor([0, 1, 2, 2], dtype=torch.int32))
    v.update(kw)
    return ps.BlockNorm(post_norm=ps.NORM_RMS, **v)


@pytest.mark.parametrize("name,field", [("post_weight", "post_weight"), ("gate", "gate"), ("mul", "mul"), ("add", "add"),
                                        ("segments", "seg_start")])
def test_a_vector_given_other_memory_is_read_there(ps, name, field):
    """By `.data`, and by a storage that is released and comes back: each call's record has the address of that time."""
    norm = vectors(ps)
    v = getattr(norm, name)
    assert getattr(norm._record(2, 8, BF16, CPU), field) == v.data_ptr()
    was = v.data_ptr()
    kept = v.data                                        # so that the allocator cannot hand out the same place again
    v.data = v.data.clone()
    assert v.data_ptr() != was and getattr(norm._record(2, 8, BF16, CPU), field) == v.data_ptr()
    assert kept.data_ptr() == was
    storage, size = v.untyped_storage(), v.untyped_storage().nbytes()
    storage.resize_(0)
    hold = [torch.empty_like(kept) for _ in range(8)]
    storage.resize_(size)
    assert getattr(norm._record(5, 8, BF16, CPU), field) == v.data_ptr() and hold


def test_a_vector_that_changed_its_kind_is_checked_again(ps):
    norm = vectors(ps)
    norm._record(2, 8, BF16, CPU)
    norm.gate.data = torch.ones(8)                       # one for all segments from now on
    rec = norm._record(2, 8, BF16, CPU)
    assert rec.flags == ps.NORM_MOD_BY_SEG and rec.gate == norm.gate.data_ptr()
    norm.gate.data = torch.ones(4, 8)
    with pytest.raises(ValueError, match="gate"):
        norm._record(2, 8, BF16, CPU)
    norm.gate.data = torch.ones(3, 8, dtype=BF16)
    with pytest.raises(ValueError, match="gate"):
        norm._record(2, 8, BF16, CPU)
    norm.gate.data = torch.ones(8, 3).t()                # the same shape in another order
    with pytest.raises(ValueError, match="gate is not contiguous"):
        norm._record(2, 8, BF16, CPU)
    norm.gate.data = torch.ones(3, 8)
    assert norm._record(2, 8, BF16, CPU).flags == ps.NORM_GATE_BY_SEG | ps.NORM_MOD_BY_SEG


def test_an_order_that_changed_in_place_is_seen(ps):
    """Address, type and shape as before, but not the strides."""
    norm = vectors(ps)
    norm._record(2, 8, BF16, CPU)
    norm.gate.as_strided_((3, 8), (1, 3))
    with pytest.raises(ValueError, match="gate is not contiguous"):
        norm._record(2, 8, BF16, CPU)


@pytest.mark.parametrize("name", ["post_weight", "gate", "mul", "add", "segments"])
def test_a_vector_without_memory_is_refused(ps, name):
    """A released storage has the address NULL, which would mean that there is no such vector."""
    norm = vectors(ps)
    norm._record(2, 8, BF16, CPU)
    v = getattr(norm, name)
    v.untyped_storage().resize_(0)
    with pytest.raises(ValueError, match=f"storage of {name} was released"):
        norm._record(2, 8, BF16, CPU)


@pytest.mark.parametrize("part", [slice(0, 4), slice(4, 8)], ids=["from the start", "with an offset"])
def test_arrays_without_memory_are_refused(ps, part):
    """Matrices and contiguous arrays, whole or parts of what was released (whose addresses are their offsets)."""
    act = ps._activations
    wide = torch.ones(4, 8)
    x, rows = wide[:, part], wide[1:3]
    assert act._matrix(x, "x", x.shape, torch.float32, CPU) == (x.data_ptr(), 8)
    assert act._whole(rows, "rows", rows.shape, act._F32, CPU) == rows.data_ptr()
    wide.untyped_storage().resize_(0)
    with pytest.raises(ValueError, match="storage of x was released"):
        act._matrix(x, "x", x.shape, torch.float32, CPU)
    with pytest.raises(ValueError, match="storage of rows was released"):
        act._whole(rows, "rows", rows.shape, act._F32, CPU)
    room = torch.ones(64, dtype=torch.uint8)[16:]
    assert act._room(room, 0, CPU, None)[1] == 48
    room.untyped_storage().resize_(0)
    with pytest.raises(ValueError, match="storage of workspace was released"):
        act._room(room, 0, CPU, None)
    empty = torch.empty(0, 8)                              # nothing to read: no memory needed
    assert act._matrix(empty, "x", empty.shape, torch.float32, CPU) == (empty.data_ptr(), 8)


def test_a_single_row_has_no_distance_to_another(ps):
    """One token's part of a matrix wider than a distance between rows may be (2^24 for dy) is a row like any other."""
    x = torch.empty(1, 1 << 25, dtype=torch.uint8)[:, 5:105]
    assert ps._activations._matrix(x, "x", x.shape, torch.uint8, CPU) == (x.data_ptr(), 100)
    x = torch.empty(2, 300, dtype=torch.uint8)[:, 5:105]
    assert ps._activations._matrix(x, "x", x.shape, torch.uint8, CPU) == (x.data_ptr(), 300)
