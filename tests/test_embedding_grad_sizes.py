"""The embedding gradient's order of a long list: work that grows with the tokens, not
with their square.  Every block of the sort walks over one row of counts for each
block, so the rows are bounded, as the workspace shows."""
from blockwise_fp8_zero_gb300 import fp8z


def _counts_bytes(tokens, vocab, hidden):
    """What the workspace holds beside keys and values (two buffers each), the pieces'
    partial sums, tickets and the rows in use: the counts, and under 2 KB of rounding up."""
    piece = 32 if tokens >= 8192 else 16 if tokens >= 2048 else 8
    pieces = -(-tokens // piece)
    rest = 16 * tokens + pieces * 2 * hidden * 4 + 3 * pieces * -(-hidden // 1024) * 4 + (vocab if tokens > 512 else 0)
    return fp8z.fp8z_embedding_grad_workspace(tokens, vocab, hidden) - rest


def test_counts_of_a_long_list_are_bounded():
    from blockwise_fp8_zero_gb300 import build
    build.build()
    row = 4096                                       # 1024 digits of 4 bytes
    for tokens in (1, 2048, 2049, 16384, 500000):
        assert _counts_bytes(tokens, 50000, 8) <= -(-tokens // 2048) * row + 2048
    for tokens in (1 << 20, (1 << 24) + 1, 1 << 28, 1 << 30):
        for vocab in (1, 50000, 1 << 30):
            assert 0 <= _counts_bytes(tokens, vocab, 8) <= 1024 * row
