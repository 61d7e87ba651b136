"""Calls of fa_qk_rope and fa_qk_rope_bwd whose tables lack rows that the tokens' own
indexes take: refused on the host.  CPU only: each call below fails a check before any
launch."""
from test_rope import A, bwd, fwd, lib          # noqa: F401  (fixtures)


def test_tables_without_a_row_for_every_token(fwd, bwd):
    """Sequences longer than the tables, whole or cut short by the number of tokens; as
    long as the tables or shorter they go on to the next check (here an alignment)."""
    for call, wrong in ((fwd, "qo"), (bwd, "dq")):
        for T, N in ((65, 65), (100, 100), (130, 65), (200, 1 << 30), (65, 2 ** 31 - 1)):
            assert call(pos=None, T=T, N=N) == -1, (T, N)
        for T, N in ((64, 64), (128, 64), (64, 1 << 30), (200, 1), (3, 4)):
            assert call(pos=None, T=T, N=N, **{wrong: 200 * A + 8}) == -3, (T, N)
        assert call(T=100, N=100, **{wrong: 200 * A + 8}) == -3          # positions decide
