"""The paged 4-bit cache's call site without a GPU: what it refuses and what it
keeps, on objects that are not constructed (a cache needs a device)."""
import pytest

torch = pytest.importorskip("torch")

NAMES = ["k_codes", "k_scale", "v_codes", "v_scale", "block_table", "seq_len", "free_list", "free_count"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from tile_routed_mixed_b200 import build
    build.build()


def _bare(**fields):
    """A cache without its device side."""
    import tile_routed_mixed_b200 as tm
    c = object.__new__(tm.TileMixKV4Cache)
    c.__dict__.update(fields)
    return c


@pytest.mark.parametrize("name", NAMES)
def test_the_tensors_cannot_be_rebound(name):
    """The kernels read and write at the addresses taken when the object was made: a
    tensor put in the place of one would never be read, and the old one's memory,
    freed, would be written."""
    x = torch.zeros(3)
    c = _bare(_tensors={name: x})
    with pytest.raises(AttributeError):
        setattr(c, name, torch.ones(3))
    assert getattr(c, name) is x
