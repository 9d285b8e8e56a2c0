"""A bounded wait of the prompt attention that runs out: every role unwinds, the call reports it and the GPU stays usable.

A test-only copy of the library has a 1 ms wait limit, and its CTA 0 never loads the values of its second step: the
issuers give up on them, the row warps on the issuers, the load warp on the ring.  All of them wait (bounded) for what
they have in flight and return; the other CTAs finish their items.  No fault, trap or hang is involved: the failure is a
load that is never issued.
"""
import ctypes
import time

import pytest
import torch

import mla_decode_attention_latent_gb300 as mla
from mla_decode_attention_latent_gb300 import _lib
from mla_decode_attention_latent_gb300 import build as cuda_build
from tests.test_prefill_gpu import check, cu_of, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rope", [True, False])
def test_a_wait_that_runs_out_is_reported(rope):
    dev, n, h = torch.device("cuda", 0), 300, 4
    lib = ctypes.CDLL(cuda_build.build_timeout_test_lib())
    for name, (res, args) in _lib.SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    mla.mla_device_status()
    q, k, v, kr = make(dev, [n], [n], h, h, rope, seed=3)
    cu = cu_of([n], dev)
    out, lse = torch.zeros((n, h, 128), dtype=torch.bfloat16, device=dev), torch.zeros((n, h), device=dev)
    ws = torch.empty((mla.mla_prefill_workspace_bytes(1, n, h, h),), dtype=torch.uint8, device=dev)
    torch.cuda.synchronize()
    t0 = time.time()
    st = lib.mla_prefill(q.data_ptr(), q.stride(0), q.stride(1), k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(), v.stride(0), v.stride(1),
                         kr.data_ptr() if rope else None, 64 if rope else 0, cu.data_ptr(), cu.data_ptr(), 1, n, n, h, h, q.shape[2], 128,
                         q.shape[2] ** -0.5, 1, None, out.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel(), torch.cuda.current_stream(dev).cuda_stream)
    assert st == _lib.MLA_OK
    status = ctypes.c_int(0)
    assert lib.mla_device_status(ctypes.byref(status), 1) == _lib.MLA_OK  # waits for the device
    elapsed = time.time() - t0
    assert status.value == _lib.MLA_DEVERR_TIMEOUT, f"status {status.value:#x}"
    assert elapsed < 30.0, f"the unwinding took {elapsed:.1f} s"
    # the longest block of head 0 is CTA 0's; the other heads are whole
    check(out, lse, q, k, v, kr, [n], [n], True, heads=[1, 2, 3])
    # the regular library, same process, same inputs
    out, lse = mla.mla_prefill(q, k, v, cu, cu, k_rope=kr)
    check(out, lse, q, k, v, kr, [n], [n], True)
    assert mla.mla_device_status() == 0
