"""The workspace that the table's gradient asks for is what the header says, at every width and number of tokens."""
import pytest


@pytest.fixture(scope="module")
def lib():
    from deterministic_token_logprob_gb300 import build
    build.build()
    import deterministic_token_logprob_gb300 as rlk
    return rlk.lib()


def stated(T, H):
    def carved(n):
        return -(-n // 256) * 256

    if T <= 256:
        return 0
    n, cut = T // 16 + 1, -(-H // 256)
    if H > 2048:
        cut = -(-H // 2048) * 8
    return 2 * carved(8 * T) + carved(16 * T + 16) + carved(8 * n * (-(-H // 8) * 8)) + carved(12 * n * cut)


def test_workspace_of_the_tables_gradient(lib):
    for H in [*range(1, 5000, 7), 256, 257, 512, 2048, 2049, 4096, 4097, 8200, 65535, 65536]:
        for T in (1, 256, 257, 300, 1000, 4097, 65536, 3000001, 1 << 24):
            assert lib.rlk_embedding_bwd_workspace(T, H) == stated(T, H), (T, H)


def test_counters_have_room_for_every_slice(lib):
    """The slices that a call counts with (1 or 2 packs a lane, up to 8 warps a CTA) are no more than the workspace has counters for."""
    for H in range(1, 65537, 3):
        room = -(-H // 256) if H <= 2048 else -(-H // 2048) * 8
        for packs in (1, 2):
            warps = min(8, -(-H // (256 * packs)))
            blocks = -(-H // (256 * packs * warps))
            assert blocks * warps <= room, (H, packs)
