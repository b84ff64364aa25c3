"""The wait by cycles of the kernels with many short waits, on a barrier that nothing arrives on: it
gives up, says so in its flag, leaves the context usable, and takes the time of its cycles."""
import pytest
import torch

from channelwise_gated_delta_gb300 import gdr_device_check
from tests.umma_diag import wait_cycles

pytestmark = pytest.mark.gpu


def test_wait_by_cycles_gives_up_in_time():
    wait_cycles()
    gave_up, seconds = wait_cycles()
    assert gave_up == 32
    # 2^24 cycles at 0.5 to 2.2 GHz, and a try's own time
    assert 2 ** 24 / 2.2e9 <= seconds <= 2 ** 24 / 0.5e9 + 0.01
    assert int((torch.ones(100, device="cuda") * 2).sum()) == 200
    gdr_device_check()
