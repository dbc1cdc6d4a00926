"""The library's calls in a context of the caller's own, and in a thread that has none."""

import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

# A host program of the driver interface: its own context, its own memory.  The weights are
# zeros: codes 8 and scales 0, and with scales of 1 a product of zeros.
OWN_CONTEXT = r"""
import ctypes as C
import sparse_moe_layer_02_b200 as moe
cu = C.CDLL("libcuda.so.1")
def ok(rc): assert rc == 0, rc
ok(cu.cuInit(0))
ctx, now = C.c_void_p(), C.c_void_p()
ok(cu.cuCtxCreate_v2(C.byref(ctx), 0, 0))
lib = moe.load_library()
def memory(n, byte):
    p = C.c_uint64()
    ok(cu.cuMemAlloc_v2(C.byref(p), C.c_size_t(n)))
    ok(cu.cuMemsetD8_v2(p, C.c_ubyte(byte), C.c_size_t(n)))
    return p.value
def read(p, n):
    b = (C.c_ubyte * n)()
    ok(cu.cuCtxSynchronize())
    ok(cu.cuMemcpyDtoH_v2(b, C.c_uint64(p), C.c_size_t(n)))
    return bytes(b)
M, K, N = 64, 256, 20
W, q, s = memory(M * K * 2, 0), memory(M * K // 2, 1), memory(K // 64 * M * 2, 1)
ok(lib.moe_quantize(W, 1, M, K, 64, q, s, None))
ok(cu.cuCtxGetCurrent(C.byref(now)))
assert now.value == ctx.value, "the call changed the current context"
assert read(q, M * K // 2) == b"\x88" * (M * K // 2) and read(s, K // 64 * M * 2) == bytes(K // 64 * M * 2)
one = memory(K // 64 * M * 2, 0x3f)
x, y = memory(N * K * 2, 0x3f), memory(N * M * 2, 1)
ok(lib.moe_linear_quant(x, q, one, N, M, K, 64, y, None))
assert read(y, N * M * 2) == bytes(N * M * 2)
ok(cu.cuCtxGetCurrent(C.byref(now)))
assert now.value == ctx.value
print("own context kept")
"""

NO_CONTEXT = r"""
import threading, torch
import sparse_moe_layer_02_b200 as moe
W = torch.randn(64, 256, device="cuda").to(torch.bfloat16)
x = torch.randn(20, 256, device="cuda").to(torch.bfloat16)
q, s = moe.moe_quantize(W, 64)
want, got = moe.moe_linear_quant(x, q, s), []
t = threading.Thread(target=lambda: got.append(moe.moe_linear_quant(x, q, s)))
t.start(); t.join()
torch.cuda.synchronize()
assert torch.equal(got[0], want)
print("thread without a context served")
"""


@pytest.mark.parametrize("program,says", [(OWN_CONTEXT, "own context kept"),
                                          (NO_CONTEXT, "thread without a context served")],
                         ids=["own", "none"])
def test_context(program, says):
    r = subprocess.run([sys.executable, "-c", program], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and says in r.stdout, r.stdout + r.stderr
