"""The output end's operators on the CPU: rules of the host side that a result
depends on, over the whole range of sizes. No GPU work."""
import pytest


@pytest.fixture(scope="module")
def zs(hip_built):
    from sharded_mixed_precision_zs_amd import zeroshard
    return zeroshard


@pytest.mark.parametrize("dtype", [0, 1, 2])
def test_parts_of_a_long_row_leave_nothing_out(zs, dtype):
    """The last part has everything from its first vector on, so that must not lie past
    the row's last one, whatever the row's alignment; the parts before it are whole.
    The workspace tells their number: 16 bytes each, and 4 a slot."""
    esz = 4 if dtype == zs.ZS_FP32 else 2
    ve = 16 // esz
    vocabs = [(16385 << s) * ve + d for s in range(8) for d in (-1, 0, 1, ve + 1, 37, 5003, 12345 * ve)]
    for rows in (1, 2, 3, 5, 7, 100, 1000, 1024, 5000):
        for vocab in [v for v in vocabs if v * esz // 16 > 512 * 32] + [349189, 698377, 1048585,
                                                                        2097165, (1 << 31) - 1]:
            if vocab * esz // 16 <= 512 * 32:
                continue
            parts, rest = divmod(zs.zs_distill_workspace(rows, vocab, 9, dtype) // rows - 36, 16)
            vecs = vocab * esz // 16
            assert rest == 0 and 1 <= parts <= vecs
            each = -(-vecs // parts)
            for head in range(ve):
                have = (vocab - head) // ve          # whole vectors after `head` elements
                assert (parts - 1) * each <= have <= parts * each


@pytest.mark.parametrize("tau,status", [(2.0 ** -127, 1), (1e-42, 1), (0.0, 1), (2.0 ** -126, 0)])
def test_a_temperature_without_a_reciprocal_is_refused(zs, tau, status):
    """rows = 0 enqueues nothing."""
    assert zs._lib.zs_distill(None, 0, 0, 100, 100, None, None, 4, tau, None, None, 1.0, None, None,
                              None, 0, None, 0, None) == status
