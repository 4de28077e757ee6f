"""Torch views of a pool's memory keep the pool, and so the memory, alive."""
import gc
import weakref

import pytest
import torch

import paged_kv_cache_19_gb300 as kp

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("which", [0, 1, 2, 3])
def test_a_view_outlives_its_pool_object(which):
    pool = kp.kv_pool_create(4, 16, 2, 64)
    view = pool.tensors()[which]
    alive = weakref.ref(pool)
    del pool
    gc.collect()
    assert alive() is not None            # before anything reads the memory
    assert torch.equal(view.float(), torch.full_like(view, 0.0 if which < 2 else 1.0).float())
    del view
    gc.collect()
    assert alive() is None


def test_raw_bytes_too():
    pool = kp.kv_pool_create(4, 16, 2, 64)
    view = pool.raw_bytes()[1][2:]
    alive = weakref.ref(pool)
    del pool
    gc.collect()
    assert alive() is not None and not view.any()
