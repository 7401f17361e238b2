"""The test hook of the products by expert takes the stalls that there are."""
from tests.test_abi_healing import EINVAL, OK, lib  # noqa: F401


def test_stalls(lib):  # noqa: F811
    for stall in (-1, 6, 1 << 30):
        assert lib.trellis_moe_experts_set_wait_test(0, stall) == EINVAL and b"stall" in lib.trellis_moe_last_error()
    for stall in range(6):
        assert lib.trellis_moe_experts_set_wait_test(1000, stall) == OK
    assert lib.trellis_moe_experts_set_wait_test(0, 0) == OK
