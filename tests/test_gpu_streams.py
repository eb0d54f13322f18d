"""Streams as callers have them: any object with a `cuda_stream` handle is a stream to every call."""
import types

import pytest
import torch

from tests.test_gpu_fast_path import CALLS, Calls, same

pytestmark = pytest.mark.gpu

NEW_OUTPUTS = {"decode": dict(out=None, lse=None), "decode_score": dict(out=None, lse=None),
               "prefill": dict(out=None, lse=None), "prefill_score": dict(out=None, lse=None),
               "rope": dict(q_out=None), "release": dict(free_count_out=None),
               "plan": dict(free_count_out=None, cu_new_lens=None, seq_lens=None, positions=None, slot_map=None)}


@pytest.mark.parametrize("compiled", [True, False])
@pytest.mark.parametrize("name", CALLS)
def test_a_stream_by_its_handle(cuda_lib, monkeypatch, name, compiled):
    fn = getattr(Calls(cuda_lib), name)
    want = fn()
    torch.cuda.synchronize()
    if not compiled:
        monkeypatch.setattr(cuda_lib, "_FAST", None)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):  # (the inputs' copies are made on this stream)
        got = fn(stream=types.SimpleNamespace(cuda_stream=st.cuda_stream), **NEW_OUTPUTS[name])
    st.synchronize()
    same(got, want)
    got = fn(stream=types.SimpleNamespace(cuda_stream=0), **NEW_OUTPUTS[name])  # the default stream
    torch.cuda.synchronize()
    same(got, want)
