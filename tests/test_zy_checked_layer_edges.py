"""The tests of the operators around layers at their edges once more, in a child process that loads the checked build:
the same results, and no violation recorded; and the tests of the norm's records."""
import pytest

from test_zy_checked_layers import test_checked_build_passes as run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["test_norm_e4m3_checked.py", "test_norm_e4m3_eps.py", "test_norm_e4m3_narrow.py", "test_norm_e4m3_waits.py",
                                  "test_layer_lists.py"])
def test_edges_under_the_checked_build(name):
    run(name)
