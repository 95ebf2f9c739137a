"""Argument checks of the paged bindings that need no GPU: CPU tensors and
wrong types are refused before the library is called."""

import pytest
import torch

import sparse_attention_csa_gb300 as csa


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def test_cpu_tensors_are_refused():
    f = torch.ones(32, dtype=torch.float64)
    with pytest.raises(TypeError):
        csa.csa_rope(bf(2, 4, 512), i32(2), f)
    with pytest.raises(TypeError):
        csa.csa_cache_append(bf(2, 512), i32(2), i32(2), i32(2, 3), bf(4, 16, 512))
    with pytest.raises(TypeError):
        csa.csa_indexer_topk_paged(bf(2, 4, 64), bf(4, 16, 64), torch.zeros(2, 4), i32(2, 3), i32(2),
                                   i32(2), 4, 8, out=i32(2, 8))
    with pytest.raises(TypeError):
        csa.csa_sparse_mla_paged(bf(2, 4, 512), bf(4, 16, 512), None, None, i32(2, 3), None, i32(2),
                                 i32(2), None, 0.05, 1, 127)


def test_wrong_kinds_are_refused():
    with pytest.raises(TypeError):
        csa.csa_sparse_mla_paged([1], bf(4, 16, 512), None, None, i32(2, 3), None, None, i32(2), None,
                                 0.05, 1, 127)
    with pytest.raises(ValueError):
        csa.csa_sparse_mla_paged(bf(4, 512), bf(4, 16, 512), None, None, i32(2, 3), None, None, i32(2),
                                 None, 0.05, 1, 127)
    with pytest.raises(TypeError):
        csa.csa_indexer_topk_paged(None, bf(4, 16, 64), None, i32(2, 3), None, i32(2), 4, 8)
