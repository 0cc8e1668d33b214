"""What the binding of the operators for activations in 8 bits holds by itself (no GPU)."""
import pytest


@pytest.fixture(scope="module")
def ss():
    import __graft_entry__
    __graft_entry__.build()
    import gaussian_splatting_differentiable_gb300 as m
    return m


@pytest.mark.parametrize("n", [0, 1, 7, 1015, 1016, 1017, 5000, (1 << 31) - 1])
@pytest.mark.parametrize("D", [1, 48, 8192, 65536])
def test_a_layer_norms_workspace_serves_both_of_its_gradients(ss, n, D):
    have = ss._layer_norm_scratch(n, D)
    assert have >= ss.ss_layer_norm_workspace_bytes(n, D) > 0
    assert have >= ss.ss_layer_norm_bwd8_workspace_bytes(n, D) > 0


def test_it_does_so_where_the_two_differ(ss, monkeypatch):
    """The gradient from kept rows may come to need more than the one from rows."""
    class Library:
        ss_layer_norm_workspace_bytes = staticmethod(lambda n, D: 1000 + n)
        ss_layer_norm_bwd8_workspace_bytes = staticmethod(lambda n, D: 5000)
    monkeypatch.setattr(ss, "_L", Library)
    assert ss._layer_norm_scratch(10, 4) == 5000 and ss._layer_norm_scratch(9000, 4) == 10000


def test_sizes_out_of_range_have_none(ss):
    assert ss._layer_norm_scratch(-1, 4) == 0 and ss._layer_norm_scratch(4, 0) == 0
