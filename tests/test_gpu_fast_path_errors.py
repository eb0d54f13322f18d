"""A CUDA error out of a call's launches reaches the caller once: the call is not made again behind it.
The error is made on the host, by a stand-in for the library's calls that launches nothing; only the
compiled path's calls go to it, the Python path has the library's own."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

STUB = r"""
// any arguments: nothing is read, so that one definition stands for every call
#define FAIL(name) int calls_##name = 0; extern "C" int name() { ++calls_##name; return 4; } \
                   extern "C" int count_##name() { return calls_##name; }
FAIL(attn_decode_paged_ex) FAIL(attn_decode_paged_score) FAIL(attn_prefill_chunk_ex)
FAIL(attn_prefill_chunk_score) FAIL(rope_append_paged) FAIL(paged_step_plan) FAIL(paged_release)
"""

CHILD = r"""
import ctypes, sys
import torch
stub = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
import long_context_paged_gb300 as pa
from tests.test_gpu_fast_path import CALLS, Calls
pa.load()
assert pa._FAST is not None
c = Calls(pa)
symbol = {"decode": "attn_decode_paged_ex", "decode_score": "attn_decode_paged_score",
          "prefill": "attn_prefill_chunk_ex", "prefill_score": "attn_prefill_chunk_score",
          "rope": "rope_append_paged", "plan": "paged_step_plan", "release": "paged_release"}
name = {"decode": "attn_decode_paged", "prefill": "attn_prefill_chunk"}
for call in CALLS:
    i32 = lambda n: torch.full((n,), 77, dtype=torch.int32, device="cuda")
    out = {"rope": ("q_out", c.qp), "plan": ("seq_lens", i32(5)), "release": ("free_count_out", i32(1))}.get(
        call, ("out", c.qd if "decode" in call else c.qp))
    mine = torch.full_like(out[1], 77)
    try:
        getattr(c, call)(**{out[0]: mine})
    except pa.PagedAttnError as e:
        assert e.code == 4 and str(e).startswith(name.get(call, symbol[call]) + " failed"), (call, str(e))
    else:
        raise AssertionError(call + ": no error was raised")
    torch.cuda.synchronize()
    assert getattr(stub, "count_" + symbol[call])() == 1, call
    assert bool((mine == 77).all()), call + " was made again"
print("all raised once")
"""


def test_a_cuda_error_is_raised_and_the_call_not_repeated(cuda_lib, tmp_path):
    (tmp_path / "stub.cpp").write_text(STUB)
    lib = str(tmp_path / "stub.so")
    subprocess.run([os.environ.get("CXX") or "g++", "-shared", "-fPIC", "-o", lib, str(tmp_path / "stub.cpp")],
                   check=True)
    r = subprocess.run([sys.executable, "-c", CHILD, lib], cwd=ROOT, env=dict(os.environ, PYTHONPATH=ROOT),
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "all raised once" in r.stdout, r.stdout[-1000:] + r.stderr[-3000:]
