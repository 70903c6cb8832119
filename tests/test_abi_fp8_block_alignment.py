"""What the decodes over the 8-bit block cache ask of their pointers: 16 bytes of rows, 4 of lengths, lambda and scales."""
import pytest
import torch

from tests.test_abi_fp8_block_host import A, CUDA, MISALIGNED, decode, lib, ptrs  # noqa: F401


@pytest.mark.parametrize("kind", ["whole", "paged", "sparse"])
def test_alignment_of_each_argument(lib, kind):                        # noqa: F811
    rows, words = (0, 1, 2, 3, 4, 10), (5, 6, 7, 8, 9)                  # q, codes, out; scales, lengths, lambda
    for i in rows:
        assert decode(lib, kind=kind, p=ptrs(11, **{f"p{i}": A + 4})) == MISALIGNED
    for i in words:
        assert decode(lib, kind=kind, p=ptrs(11, **{f"p{i}": A + 2})) == MISALIGNED
        if not torch.cuda.is_available():
            assert decode(lib, kind=kind, p=ptrs(11, **{f"p{i}": A + 4})) == CUDA
