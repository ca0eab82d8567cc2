"""Sizes that the C ABI's 32-bit integers cannot hold (no GPU: tensors without memory, a library that must not be
reached)."""
import types

import pytest
import torch

from paged_kv_chunk_gb300 import capi

FAR = 2 ** 32 + 16      # as a C int: 16


def meta(*shape, dtype):
    return torch.empty(shape, dtype=dtype, device="meta")


@pytest.fixture()
def unreachable(monkeypatch):
    def call(*args):
        raise AssertionError("the library was called")

    names = [n for n in capi.header_symbols() if n.startswith("oasr_")]
    monkeypatch.setattr(capi, "_good", lambda *a: True)
    monkeypatch.setattr(capi, "_lib_device", lambda: (types.SimpleNamespace(**{n: call for n in names}), 0))


@pytest.mark.parametrize("M,K", [(FAR, 16), (3, FAR)])
def test_quantize_rows(unreachable, M, K):
    with pytest.raises(ValueError, match="2\\^31"):
        capi.oasr_quantize_rows(meta(M, K, dtype=torch.bfloat16), stream=0)


@pytest.mark.parametrize("M,N,K", [(FAR, 8, 16), (8, FAR, 16), (8, 8, FAR)])
def test_linear(unreachable, M, N, K):
    i8, f32 = torch.int8, torch.float32
    with pytest.raises(ValueError, match="2\\^31"):
        capi.oasr_linear_w8a8(meta(M, K, dtype=i8), meta(M, dtype=f32), meta(N, K, dtype=i8), meta(N, dtype=f32), stream=0)


@pytest.mark.parametrize("M,R", [(FAR, 31), (16, FAR)])
def test_project(unreachable, M, R):
    i8, f32 = torch.int8, torch.float32
    with pytest.raises(ValueError, match="2\\^31"):
        capi.oasr_project_qkv_pos_w8a8(meta(M, 64, dtype=i8), meta(M, dtype=f32), meta(192, 64, dtype=i8), meta(192, dtype=f32),
                                       meta(192, dtype=torch.bfloat16), meta(R, 64, dtype=i8), meta(R, dtype=f32),
                                       meta(64, 64, dtype=i8), meta(64, dtype=f32), 1, stream=0)


@pytest.mark.parametrize("width,length", [(FAR, 16), (4, FAR)])
def test_cache(unreachable, width, length):
    pool, scale = meta(4, 1, 16, 64, dtype=torch.float8_e4m3fn), meta(4, 1, 2, 16, dtype=torch.uint8)
    table, lens = meta(1, width, dtype=torch.int32), meta(1, dtype=torch.int32)
    new = meta(1, 2, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="2\\^31"):
        capi.oasr_paged_read_e4m3(pool, pool, scale, table, lens, length, stream=0)
    if width == FAR:
        with pytest.raises(ValueError, match="2\\^31"):
            capi.oasr_paged_append_e4m3(new, new, pool, pool, scale, table, lens, stream=0)
