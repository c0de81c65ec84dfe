"""The cross entropy's workspaces at the row counts where their stated limits change."""
import pytest

import speculative_decoding_verification_83_gb300 as dv

V = 248320


@pytest.fixture(scope="module")
def lib():
    dv.build()
    return dv.load()


def up(n):
    return (n + 255) // 256 * 256


@pytest.mark.parametrize("rows", [1, 33, 1000, 16384, 65535, 65536, 65537, 70001, 1 << 17, 1 << 20])
@pytest.mark.parametrize("K", [64, 1024])
def test_a_piece_of_the_logits_gradients(lib, rows, K):
    """One piece: 512 MiB at most, and 8 KiB a row beyond 2^16 rows; a copy of the hidden states, dh in fp32 up to 8
    times (runs of 32 rows), and 24 bytes a row."""
    have = lib.dflash_linear_entropy_workspace_bytes(rows, V, K, 1)
    piece = up(max(512 << 20, 8192 * rows) if rows > 1 << 16 else 512 << 20)
    most = piece + up(rows * K * 2) + 8 * up((rows + 31) // 32 * 32 * K * 4) + 24 * rows + 5 * 256
    assert have <= most
    if rows >= 1 << 16:  # (and not much less)
        assert have >= 8192 * rows + rows * K * 2
    if rows > 1 << 16:
        assert have > 512 << 20
