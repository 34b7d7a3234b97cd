"""Scalars of the shared-prompt calls: whatever converts to a number is taken,
as by the other calls (CPU only; the library is a stand-in)."""
import types

import numpy as np
import pytest
import torch

from paged_mla_speculative_gb300 import binding as mb

I32, BF = torch.int32, torch.bfloat16


class _Library:
    """Converts arguments as ctypes does, and returns MLA_VERIFY_OK."""

    def __getattr__(self, name):
        types_ = mb.SIGNATURES[name][1]

        def call(*args):
            for t, a in zip(types_, args):
                t.from_param(a)
            self.args = args
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    lib = _Library()
    monkeypatch.setattr(mb, "load_library", lambda: lib)
    monkeypatch.setattr(mb, "_stream_ptr", lambda stream: 0)
    return lib


def _plan():
    return types.SimpleNamespace(torch_device=torch.device("cpu"), num_slots=128, H=2, T=4, max_kv_len=100, page_size=64,
                                 out_dtype=torch.float32, handle=None)


@pytest.mark.parametrize("x", [0.25, np.float32(0.25), np.float64(0.25), torch.tensor(0.25)])
def test_scale_and_eps(lib, x):
    z = lambda *s: torch.zeros(s, dtype=I32)  # noqa: E731
    cache = torch.zeros(128, 576, dtype=BF)
    mb.mla_verify_attn_shared(_plan(), torch.zeros(1, 4, 2, 576, dtype=BF), cache, z(2), z(2), z(1), z(1, 4), x, z(2), z(1),
                              out=torch.zeros(1, 4, 2, 512), lse=torch.zeros(1, 4, 2))
    assert lib.args[8] == 0.25
    mb.append_kv(_plan(), torch.zeros(3, 576, dtype=BF), torch.zeros(512, dtype=BF), x, torch.zeros(8, 64), z(3), z(3), cache)
    assert lib.args[5] == 0.25


@pytest.mark.parametrize("x", [3, np.int32(3), np.int64(3), torch.tensor(3)])
def test_extra_rows(lib, x):
    z = lambda n: torch.zeros(n, dtype=I32)  # noqa: E731
    mb.fork_kv(_plan(), z(3), z(4), z(3), z(2), torch.zeros(128, 576, dtype=BF), z(2), z(2), z(1), x)
    assert lib.args[10] == 3
