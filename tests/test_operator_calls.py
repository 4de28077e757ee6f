"""CPU checks of the norm-rotation-append, masked and shared-prefix calls: declared, exported,
and refused on the host; groups of sequences that share blocks, from the block manager."""
import ctypes
import os

import pytest

import paged_kv_cache_19_gb300 as kp
from paged_kv_cache_19_gb300 import build as cuda_build

HEADERS = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    return kp.load_library()


def test_declared_exported_and_bound(lib):
    text = "".join(open(os.path.join(HEADERS, f)).read() for f in os.listdir(HEADERS))
    for name in ("paged_norm_rope_append", "paged_attention_masked", "paged_attention_masked_workspace_size",
                 "paged_shared_prefix_attention", "paged_shared_prefix_workspace_size"):
        assert f"kv_status {name}(" in text and hasattr(lib, name) and callable(getattr(kp, name)) and name in kp.__all__
    assert "kv_status kv_bm_prefix_groups(" in text and "KV_DEVERR_GROUP    0x20u" in text and kp.DEVERR_GROUP == 0x20


def test_a_null_pool_is_refused(lib):
    bad = kp.KV_ERR_INVALID_ARG
    n = ctypes.c_size_t()
    assert lib.paged_norm_rope_append(None, 16, 64, 16, 64, 16, 64, 1, 1, None, None, 0.0, None, 0, 0, 0, None, None, 16, 1,
                                      16, 1, 1, 16, None) == bad
    assert lib.paged_attention_masked(None, 16, 1, 1, 16, 1, 16, 1, 1.0, None, 0, None, 0, 16, None, None) == bad
    assert lib.paged_attention_masked_workspace_size(None, 1, 1, 1, 1, 0, 0, ctypes.byref(n)) == bad
    assert lib.paged_shared_prefix_attention(None, 16, 1, 1, 16, 1, 16, 1, None, None, 0, 1.0, 0, None, 0, 16, None,
                                             None) == bad
    assert lib.paged_shared_prefix_workspace_size(None, 1, 1, 1, 1, 0, 0, ctypes.byref(n)) == bad
    assert lib.paged_shared_prefix_workspace_size(None, 1, 1, 1, 1, 0, 0, None) == bad


def test_host_tensors_are_refused(lib):
    """The native binding looks at every tensor before it calls the library."""
    import torch
    c = kp._native()
    q, kv = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    t, l = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)  # noqa: E741
    out = torch.empty_like(q)
    for call, args in ((c.norm_rope_append, (1, 64, 2, q, kv, kv, t, l, None, None, 1e-6, None, False, 1, None, None, out, 0)),
                       (c.attention_masked, (1, 64, q, t, l, 1.0, 0.0, 0, None, None, None, 0, None, out, None, 0)),
                       (c.shared_prefix_attention, (1, 64, q, t, l, l, l[:1], 1.0, 0, None, out, None, 0))):
        with pytest.raises(ValueError, match="CUDA"):
            call(*args)
        with pytest.raises(RuntimeError, match="destroyed"):
            call(None, *args[1:])
        with pytest.raises(TypeError):
            call(*args[:-1])
        with pytest.raises(ValueError, match="tensor"):
            call(*args[:2], *[None if isinstance(x, torch.Tensor) else x for x in args[2:]])
        with pytest.raises(ValueError):
            call(*args[:1], 128, *args[2:])


def test_tensors_without_plain_memory_are_refused(lib):
    """Sparse, meta and fake tensors make torch throw below the binding; sizes past 32 bits do not
    fit the C ABI.  Meta tensors stand in for the large ones."""
    import torch
    c = kp._native()
    q, kv = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    t, l = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)  # noqa: E741
    out = torch.empty_like(q)
    calls = ((c.norm_rope_append, (1, 64, 2, q, kv, kv, t, l, None, None, 1e-6, None, False, 1, None, None, out, 0)),
             (c.attention_masked, (1, 64, q, t, l, 1.0, 0.0, 0, None, None, None, 0, None, out, None, 0)),
             (c.shared_prefix_attention, (1, 64, q, t, l, l, l[:1], 1.0, 0, None, out, None, 0)))
    for call, args in calls:
        for odd in (lambda x: x.to("meta"), lambda x: x.to_sparse(), lambda x: x.to(torch.float32).to_sparse()):
            with pytest.raises(ValueError):
                call(*[odd(x) if isinstance(x, torch.Tensor) else x for x in args])
            for i, x in enumerate(args):
                if isinstance(x, torch.Tensor):
                    with pytest.raises(ValueError):
                        call(*args[:i], odd(x), *args[i + 1:])
        wide = torch.empty(2, 2 ** 32 + 3, dtype=torch.int32, device="meta")
        with pytest.raises(ValueError, match="2.31|CUDA"):
            call(*[wide if x is t else x for x in args])


def groups(bm, seqs, **kw):
    order, off, blk = (t.tolist() for t in bm.prefix_groups(seqs, **kw))
    assert sorted(order) == list(range(len(seqs))) and off[0] == 0 and off[-1] == len(seqs) and len(off) == len(blk) + 1
    return [([seqs[i] for i in order[off[g]:off[g + 1]]], blk[g]) for g in range(len(blk))]


def test_groups_of_forks_and_cached_prompts():
    bm = kp.BlockManager(64, 4, prefix_caching=True)
    prompt = list(range(11))
    bm.add_sequence(1)
    bm.append_slots(1, 11, prompt)                    # two full blocks and three tokens
    bm.fork(1, 2)
    bm.add_sequence(3)
    bm.append_slots(3, 9, [7] * 9)
    bm.add_sequence(4)                                # the same prompt through the prefix cache
    assert bm.match_prefix(4, prompt) == 8
    bm.append_slots(4, 3, prompt[8:])
    bm.add_sequence(5)                                # one block in common
    assert bm.match_prefix(5, prompt[:4] + [99] * 6) == 4
    bm.append_slots(5, 6, [99] * 6)
    bm.add_sequence(6)                                # empty
    assert groups(bm, [3, 1, 6, 2, 4, 5]) == [([3], 0), ([1, 2, 4, 5], 1), ([6], 0)]
    assert groups(bm, [3, 1, 6, 2, 4, 5], min_blocks=2) == [([3], 0), ([1, 2, 4], 2), ([6], 0), ([5], 0)]
    assert groups(bm, [3, 1, 6, 2, 4, 5], min_blocks=3) == [([s], 0) for s in (3, 1, 6, 2, 4, 5)]
    # the partly filled last block of the forks is shared too, but not full: it never counts,
    # also when it is full in one of them
    bm.append_slots(2, 1, [11])
    assert groups(bm, [2, 1]) == [([2, 1], 2)]
    assert groups(bm, []) == []
    bm.close()


def test_the_same_sequence_twice_is_a_group():
    bm = kp.BlockManager(8, 4)
    bm.add_sequence(1)
    bm.append_slots(1, 8)
    assert groups(bm, [1, 1]) == [([1, 1], 2)]
    bm.close()


def test_groups_refusals(lib):
    bm = kp.BlockManager(8, 4)
    bm.add_sequence(1)
    with pytest.raises(kp.KVError):
        bm.prefix_groups([1, 2])
    with pytest.raises(kp.KVError):
        bm.prefix_groups([1], min_blocks=0)
    n = ctypes.c_int()
    assert lib.kv_bm_prefix_groups(None, None, 0, 1, None, None, None, ctypes.byref(n)) == kp.KV_ERR_INVALID_ARG
    assert lib.kv_bm_prefix_groups(bm._h, None, 1, 1, None, None, None, ctypes.byref(n)) == kp.KV_ERR_INVALID_ARG
    bm.close()


@pytest.mark.parametrize("shape", [(0, 64), (5, 0), (0, 0), (64,)])
def test_a_rotation_table_without_rows_is_refused(lib, shape):
    """Its address is null, which the C call takes for "no rotation"."""
    import torch
    q, kv = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    t, l = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)  # noqa: E741
    with pytest.raises(ValueError, match="rope_table"):
        kp._native().norm_rope_append(1, 64, 2, q, kv, kv, t, l, None, None, 1e-6, torch.zeros(shape), False, 1, None, None,
                                      torch.empty_like(q), 0)


def test_an_argument_without_a_truth_value_is_refused(lib):
    """The error of its conversion is the call's error (the call went on with the error set)."""
    import torch
    q, kv = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    t, l = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)  # noqa: E741
    with pytest.raises(RuntimeError, match="ambiguous"):
        kp._native().norm_rope_append(1, 64, 2, q, kv, kv, t, l, None, None, 1e-6, None, torch.zeros(2), 1, None, None,
                                      torch.empty_like(q), 0)


def test_fake_tensors_are_refused(lib):
    """They have a CUDA device and no memory: one in the place of an optional tensor (a rotation
    table, a log-sum-exp) was taken for none, and all of them together for a call of null pointers."""
    import torch
    from torch._subclasses.fake_tensor import FakeTensorMode
    c = kp._native()

    def fake(t):
        with FakeTensorMode():
            return torch.empty(t.shape, dtype=t.dtype, device="cuda:0")

    q, kv = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    t, l = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)  # noqa: E741
    out, w, table = torch.empty_like(q), torch.zeros(64), torch.zeros(9, 64)
    ws, lse = torch.zeros(64, dtype=torch.uint8), torch.zeros(2, 4)
    for call, args in ((c.norm_rope_append, (1, 64, 2, q, kv, kv, t, l, w, w, 1e-6, table, False, 1, None, None, out, 0)),
                       (c.attention_masked, (1, 64, q, t, l, 1.0, 0.0, 0, w[:4], l, l, 0, ws, out, lse, 0)),
                       (c.shared_prefix_attention, (1, 64, q, t, l, t[0], l[:2], 1.0, 0, ws, out, lse, 0))):
        with pytest.raises(ValueError, match="memory"):
            call(*[fake(x) if isinstance(x, torch.Tensor) else x for x in args])


def test_tensors_of_two_devices_are_refused(lib):
    """A kernel must not be given an address of another device than its pool's.  Fake tensors stand in
    for the devices."""
    import torch
    if torch.cuda.is_available() and torch.cuda.device_count() < 2:
        pytest.skip("a fake tensor of a second device wants one, or no device at all")
    from torch._subclasses.fake_tensor import FakeTensorMode
    c = kp._native()

    def fake(t, device):
        with FakeTensorMode():
            return torch.empty(t.shape, dtype=t.dtype, device=device)

    q, kv = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    t, l = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)  # noqa: E741
    out, w, table = torch.empty_like(q), torch.zeros(64), torch.zeros(9, 64)
    ws, lse = torch.zeros(64, dtype=torch.uint8), torch.zeros(2, 4)
    for call, args in ((c.norm_rope_append, (1, 64, 2, q, kv, kv, t, l, w, w, 1e-6, table, False, 1, l, l, out, 0)),
                       (c.attention_masked, (1, 64, q, t, l, 1.0, 0.0, 0, w[:4], l, l, 0, ws, out, lse, 0)),
                       (c.shared_prefix_attention, (1, 64, q, t, l, l, l[:1], 1.0, 0, ws, out, lse, 0))):
        for other in [i for i, x in enumerate(args) if isinstance(x, torch.Tensor)]:
            with pytest.raises(ValueError, match="one device"):
                call(*[fake(x, "cuda:1" if i == other else "cuda:0") if isinstance(x, torch.Tensor) else x
                       for i, x in enumerate(args)])
