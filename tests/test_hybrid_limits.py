"""The launch limits that gdn_hybrid.h states, at their ends (CPU: size queries answer 0 for an invalid problem)."""
import pytest

A = 0x10000  # an aligned address that is never read


@pytest.fixture(scope="module")
def G():
    import gated_delta_rule_34_amd as G

    return G


def glr(G, N, T_total, channels, dtype, table):
    p = G.gdn_glr_problem(N=N, T=0 if table or not N else T_total // N, T_total=T_total, channels=channels, dtype=dtype, rate=8.0, cu_seqlens=A if table else None)
    setattr(p, "lambda", A)
    return G.gdn_glr_state_bytes(p) > 0


@pytest.mark.parametrize("table", [False, True])
@pytest.mark.parametrize("bf16", [False, True])
def test_recurrence_takes_what_the_header_says(G, table, bf16):
    """(N + 1) ceil(channels / 32) + 512 up to 2^23, channels below 2^23 bytes, rows up to 2^28; N past 2^23 never."""
    dtype, size = (G.GDN_BF16, 2) if bf16 else (G.GDN_F32, 4)
    for channels in (8, 24, 32, 40, 2560, 4096, 65544, (1 << 23) // size - 8):
        N = ((1 << 23) - 512) // -(-channels // 32) - 1
        for total in (0, N, N * 31, (1 << 28) // N * N):
            assert glr(G, N, total, channels, dtype, table), (N, total, channels)
        assert not glr(G, 1 << 23, 0, channels, dtype, table) and not glr(G, 1 << 23, 1 << 23, channels, dtype, table)
    for channels in ((1 << 23) // size, 1 << 23, 1 << 28, 2**31 - 8):
        assert not glr(G, 1, 0, channels, dtype, table) and not glr(G, 1, 1, channels, dtype, table), channels
