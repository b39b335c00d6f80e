"""Paged pools, block tables and logical views for the tests of the paged operators."""

from __future__ import annotations

from typing import List, Tuple

import torch

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def block_table(lengths: List[int], page: int, seed: int, spare: int = 3) -> Tuple[torch.Tensor, int]:
    """Shuffled pages for sequences of these many positions; entries behind a
    sequence's last page hold an id outside the pool (they may not be read).
    Returns the table [B][max_blocks] and the number of pages."""
    g = torch.Generator().manual_seed(seed)
    blocks = [-(-n // page) for n in lengths]
    num = sum(blocks) + spare
    order = torch.randperm(num, generator=g).tolist()
    table = torch.full((len(lengths), max(max(blocks), 1) + 1), 1 << 30, dtype=torch.int32)
    for b, n in enumerate(blocks):
        for i in range(n):
            table[b, i] = order.pop()
    return table, num


def pool(num: int, Hkv: int, page: int, D: int, dtype: torch.dtype, seed: int) -> torch.Tensor:
    g = torch.Generator().manual_seed(seed)
    return torch.randn(num, Hkv, page, D, generator=g).to(dtype)


def logical(pages: torch.Tensor, row: torch.Tensor, n: int) -> torch.Tensor:
    """Positions 0 .. n-1 of one sequence as [Hkv][n][D] (row: its block table)."""
    page = pages.shape[2]
    pos = torch.arange(n)
    return pages[row.long()[pos // page], :, pos % page].transpose(0, 1)


def raw(t: torch.Tensor) -> torch.Tensor:
    """The bits, so that NaN compares equal to itself."""
    return t.view(torch.int16) if t.dtype == torch.bfloat16 else t.view(torch.int32)
