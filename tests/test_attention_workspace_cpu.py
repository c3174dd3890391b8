"""spec_attention_workspace_bytes gives 0 for every size that the call refuses (CPU only)."""
import pytest

from speculative_decoding_verification_34_gb300 import build
from speculative_decoding_verification_34_gb300 import specverify as sv


@pytest.fixture(scope="module", autouse=True)
def lib():
    return sv.load_library(build.build())


@pytest.mark.parametrize("Hq,Hkv", [(1025, 1), (2 ** 31 - 1, 1), (2 ** 25, 1), (2050, 2), (2 ** 26 + 2 ** 20, 2 ** 10), (1025, 1025)])
@pytest.mark.parametrize("gmax", [0, 4, 63])
def test_groups_and_heads_beyond_the_limits(Hq, Hkv, gmax):
    assert sv.spec_attention_workspace_bytes(1, gmax, Hq, Hkv, 128) == 0


def test_the_largest_sizes_have_one():
    most = sv.spec_attention_workspace_bytes(1, 63, 64, 1, 128)
    for Hq, Hkv in ((1024, 1), (1024 * 1024, 1024), (1024, 1024)):
        assert 0 < sv.spec_attention_workspace_bytes(1, 63, Hq, Hkv, 128) <= most
