"""Layouts for the checks of test_gpu_residual_norm: there every output starts beside a 16-byte boundary."""
from block_harness import Guarded


class Aligned(Guarded):
    """Guarded, with rows on 16-byte boundaries (for widths that are multiples of 8)."""

    def __init__(self, rows, cols, dtype, pad=0, offset=0, like=None):
        super().__init__(rows, cols, dtype, (pad + 7) // 8 * 8, 0, like)
