"""Refusals of the paged operators' binding that need no GPU: arguments that the
entry points would read with other strides or types than the tensors have."""
import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_11_b200 import build
    build.build()
    from sparse_attention_11_b200 import dsa
    return dsa


def test_indexer_args_layouts(lib):
    table = torch.zeros(2, 2, dtype=torch.int32)
    codes = lib.Pages(table, idx=torch.zeros(4, 16, 128, dtype=torch.uint8), idx_scale=torch.zeros(4, 16))
    plain = lib.Pages(table, idx=torch.zeros(4, 16, 128))
    q8, s, w8 = torch.zeros(6, 128, dtype=torch.uint8), torch.zeros(6), torch.zeros(128, 128, dtype=torch.bfloat16)
    q, w, k = torch.zeros(6, 128), torch.zeros(128, 128), torch.zeros(6, dtype=torch.int32)
    lib.paged_indexer_args(codes, q8, s, w8, k)
    lib.paged_indexer_args(plain, q, None, w, k)
    bad = [
        lambda: lib.paged_indexer_args(codes, torch.zeros(6, 256, dtype=torch.uint8)[:, :128], s, w8),
        lambda: lib.paged_indexer_args(codes, torch.zeros(6, 64, dtype=torch.uint8), s, w8),
        lambda: lib.paged_indexer_args(codes, q8[::2], s, w8),
        lambda: lib.paged_indexer_args(codes, q8, None, w8),
        lambda: lib.paged_indexer_args(codes, q8, s[:5], w8),
        lambda: lib.paged_indexer_args(codes, q8, s.double(), w8),
        lambda: lib.paged_indexer_args(codes, q8, torch.zeros(6, 2)[:, 0], w8),
        lambda: lib.paged_indexer_args(codes, q8, s, w),
        lambda: lib.paged_indexer_args(codes, q8, s, w8.T),
        lambda: lib.paged_indexer_args(codes, q8, s, w8[:64]),
        lambda: lib.paged_indexer_args(codes, q8, s, w8, k.long()),
        lambda: lib.paged_indexer_args(codes, q8, s, w8, k[:5]),
        lambda: lib.paged_indexer_args(codes, q8, s, w8, torch.zeros(12, dtype=torch.int32)[::2]),
        lambda: lib.paged_indexer_args(plain, q, s, w),
        lambda: lib.paged_indexer_args(plain, q, None, w8),
        lambda: lib.paged_indexer_args(plain, torch.zeros(128, 6).T, None, w),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"accepted: {i}")
