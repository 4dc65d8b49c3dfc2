"""The selective scan with a group a channel, as many of them as fill more than one
launch of the column sums."""
import pytest

from tests.ssm_util import make_scan
from tests.test_gpu_scan import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [40, 1 << 17])
def test_a_group_a_channel(D):
    """A group takes 64 columns of 16 states: 2^17 of them are 2^22 workgroups of 1024
    threads, one launch's limit."""
    check(make_scan(1600, 1, 2, D, 16, D, "bf16"))
