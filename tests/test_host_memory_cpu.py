"""Tests that let a call on host memory go on to its launch are skipped where
there is a GPU to launch it."""

import types

import pytest
import torch

import conftest


@pytest.mark.parametrize("gpu", [False, True])
def test_modules_of_host_memory_are_skipped_with_a_gpu(gpu, monkeypatch):
    monkeypatch.setattr(torch.cuda, "is_available", lambda: gpu)
    for name in ("test_abi_operators_cpu", "test_cache_overlap_cpu"):
        item = types.SimpleNamespace(module=types.SimpleNamespace(__name__=name))
        if gpu:
            with pytest.raises(pytest.skip.Exception):
                conftest.pytest_runtest_setup(item)
        else:
            conftest.pytest_runtest_setup(item)
    conftest.pytest_runtest_setup(types.SimpleNamespace(module=types.SimpleNamespace(__name__="test_abi_cpu")))
