"""The most query heads of a rotary append (no device work)."""
from test_rows_args import desc, lib, rotary  # noqa: F401 (lib is a fixture)


def test_query_channels_of_a_token_are_bounded(lib):  # noqa: F811
    most = (1 << 30) // 128
    c = desc(B=1)
    # (ws of no bytes: the call ends at the workspace's check)
    assert rotary(lib, c, n=1, Q=0x700, Qo=0x700, H_q=most, nb=0) == 6
    assert rotary(lib, c, n=1, Q=0x700, Qo=0x700, H_q=most + 1, nb=0) == 2 and b"H_q" in lib.kv2_last_error()
    assert rotary(lib, desc(B=1, d=64), n=1, rot=64, Q=0x700, Qo=0x700, H_q=2 * most, nb=0) == 6
    assert rotary(lib, c, n=1, H_q=most + 1, nb=0) == 6            # no queries: their number is not looked at
