"""A refusal of the binding that goes by a tensor's number of dimensions: nothing of the call runs."""
import pytest

from tests import test_binding_devices as devices
from tests.test_abi_expert_training import B, CALLS, F32, OnGpu
from tests.test_abi_moe_layer import lib  # noqa: F401  (the fixture)
from tests.test_binding_devices import hg  # noqa: F401  (the fixture)


def test_rows_of_more_than_one_dimension_are_refused(hg, monkeypatch):  # noqa: F811
    record = devices.Recorder()
    monkeypatch.setattr(hg.lib, "hg_grouped_wgrad", record)
    dy, _, off, _, workspace = CALLS["hg_grouped_wgrad"][1]
    # [9, 8, 9] would be taken for rows of 8, though the next row is 72 elements on
    with pytest.raises(AssertionError):
        hg.hg_grouped_wgrad(OnGpu(*dy, 0), OnGpu((9, 8, 9), B, 0), OnGpu(*off, 0),
                            dw=OnGpu((2, 64, 8), F32, 0), workspace=OnGpu(*workspace, 0))
    assert not record.calls
