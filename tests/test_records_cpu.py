"""The binding's extension: gdp_tensor records of torch tensors (host tensors here), against the ctypes
marshalling, and its refusals."""
import ctypes
import os

import pytest
import torch

from gated_deltaproduct_recurrence_amd import binding, build
from gated_deltaproduct_recurrence_amd._records import records


def same(record, tensor):
    want = binding.as_gdp_tensor(tensor)
    got = binding.gdp_tensor.from_address(record)
    assert (got.data, got.dtype, got.ndim) == (want.data, want.dtype, want.ndim)
    n = tensor.dim()
    assert list(got.shape)[:n] == list(tensor.shape) and list(got.stride)[:n] == list(tensor.stride())


def test_records_equal_the_ctypes_marshalling():
    wide = torch.zeros(5, 4, 6, 8)
    tensors = [torch.zeros(3), torch.zeros(2, 3, dtype=torch.bfloat16), wide, wide[:, 1:3, ::2], wide[0, 0, 0, 0],
               torch.zeros(4, dtype=torch.int64), torch.zeros(0, 7, dtype=torch.float16),
               torch.zeros(1, 6, dtype=torch.int32).expand(5, 6), torch.zeros(3, requires_grad=True)]
    got = records(-1, *tensors)
    assert len(got) == len(tensors) + 1 and isinstance(got[-1], bytes)
    for record, tensor in zip(got, tensors):
        same(record, tensor)
    assert len(set(got[:-1])) == len(tensors)


def test_absent_tensors_are_none():
    t = torch.zeros(2)
    got = records(-1, None, t, None)
    assert got[0] is None and got[2] is None
    same(got[1], t)


def test_two_calls_do_not_share_records():
    a, b = torch.zeros(2, 3), torch.zeros(4)
    ra, rb = records(-1, a), records(-1, b)
    same(ra[0], a)
    same(rb[0], b)


def test_refusals():
    with pytest.raises(ValueError, match="expected a tensor on cuda:0, got one on cpu"):
        records(0, torch.zeros(2))
    with pytest.raises(ValueError, match="unsupported dtype"):
        records(-1, torch.zeros(2, dtype=torch.float64))
    with pytest.raises(ValueError, match="at most 4 dims"):
        records(-1, torch.zeros(1, 1, 1, 1, 1))
    with pytest.raises(TypeError, match="torch.Tensor or None"):
        records(-1, [1.0])
    with pytest.raises(ValueError, match="negated"):
        records(-1, torch.zeros(3, dtype=torch.complex64).conj().imag)
    with pytest.raises(TypeError):
        records()
    with pytest.raises((ValueError, RuntimeError)):
        records(-1, torch.zeros(2).to_sparse())


def test_source_exists():
    assert os.path.isfile(build.RECORDS_SOURCE)


def test_record_size():
    """An extension that was built against another gdp_tensor is not used (tests/test_import_cpu.py)."""
    from gated_deltaproduct_recurrence_amd import _records
    assert _records.record_bytes == ctypes.sizeof(binding.gdp_tensor)
    one, two = records(-1, torch.zeros(2), torch.zeros(2))[:2]
    assert two - one == _records.record_bytes
