"""The products in a second context of the same GPU, plain and captured as that context's first call, and after
the first context has been taken down and made again: a kernel's limit of shared memory, set once per
device, holds in all of them."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

COMMON = r"""
import ctypes
import torch
import combine_layout_02_gb300 as ep

ROWS, E, K, F = 700, 2, 256, 512          # tiles with more shared memory than a launch has unasked
gen = torch.Generator().manual_seed(1)
host = [torch.randint(-2, 3, s, generator=gen).to(torch.bfloat16) for s in ((ROWS, K), (E, F, K), (E, 2 * F, K))]
host.append(torch.tensor([0, 300, ROWS], dtype=torch.int32))
shape = ep.ep_gemm_shape(ROWS, E, K, F)

def calls(x, w, both, prefix, y, h, launch):
    ep.ep_expert_gemm(shape, x, w, prefix, y, launch)
    ep.ep_expert_gated(shape, x, both, prefix, ep.EP_ACT_SILU, h, None, launch)

cu = ctypes.CDLL("libcuda.so.1")
P, Z, U64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_uint64
cu.cuMemAlloc_v2.argtypes = [ctypes.POINTER(U64), Z]
cu.cuMemFree_v2.argtypes = [U64]
cu.cuMemcpyHtoD_v2.argtypes = [U64, P, Z]
cu.cuMemcpyDtoH_v2.argtypes = [P, U64, Z]
cu.cuStreamCreate.argtypes = [ctypes.POINTER(P), ctypes.c_uint]
cu.cuStreamBeginCapture_v2.argtypes = [P, ctypes.c_int]
cu.cuStreamEndCapture.argtypes = [P, ctypes.POINTER(P)]
cu.cuGraphInstantiateWithFlags.argtypes = [ctypes.POINTER(P), P, ctypes.c_ulonglong]
cu.cuGraphLaunch.argtypes = [P, P]
cu.cuStreamSynchronize.argtypes = [P]
cu.cuCtxSetCurrent.argtypes = [P]
cu.cuCtxDestroy_v2.argtypes = [P]

def ok(status):
    assert status == 0, status

def put(t):          # in the current context's memory
    p, n = U64(), t.numel() * t.element_size()
    ok(cu.cuMemAlloc_v2(ctypes.byref(p), n))
    ok(cu.cuMemcpyHtoD_v2(p.value, t.data_ptr(), n))
    return ep._Address(p.value)

def put_all():
    return [put(t) for t in host] + [put(torch.zeros(ROWS, F, dtype=torch.bfloat16)) for _ in range(2)]

def results(args):
    out = [torch.empty(ROWS, F, dtype=torch.bfloat16) for _ in range(2)]
    for t, at in zip(out, args[-2:]):
        ok(cu.cuMemcpyDtoH_v2(t.data_ptr(), int(at), t.numel() * 2))
    return out
"""

SECOND = COMMON + r"""
# in the first context
dev = [t.cuda() for t in host]
out = [torch.zeros(ROWS, F, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
calls(*dev, *out, ep.make_launch())
torch.cuda.synchronize()
want = [t.cpu() for t in out]

def in_a_context_of_its_own(captured):
    ctx, stream = P(), P()
    ok(cu.cuCtxCreate_v2(ctypes.byref(ctx), 0, 0))          # current from here on
    ok(cu.cuStreamCreate(ctypes.byref(stream), 0))
    args = put_all()
    launch = ep.ep_launch(stream.value, None, None, None)
    if captured:
        graph, run = P(), P()
        ok(cu.cuStreamBeginCapture_v2(stream, 2))          # relaxed
        calls(*args, launch)
        ok(cu.cuStreamEndCapture(stream, ctypes.byref(graph)))
        ok(cu.cuGraphInstantiateWithFlags(ctypes.byref(run), graph, 0))
        for _ in range(2):
            ok(cu.cuGraphLaunch(run, stream))
    else:
        calls(*args, launch)
        calls(*args, launch)
    ok(cu.cuStreamSynchronize(stream))
    assert all(torch.equal(a, w) for a, w in zip(results(args), want))
    for at in args:
        ok(cu.cuMemFree_v2(int(at)))
    ok(cu.cuCtxDestroy_v2(ctx))

for captured in CAPTURED:
    in_a_context_of_its_own(captured)
    # and the first context's calls are as they were
    again = [torch.zeros_like(t) for t in out]
    calls(*dev, *again, ep.make_launch())
    torch.cuda.synchronize()
    assert all(torch.equal(a.cpu(), w) for a, w in zip(again, want))
print("fine")
"""

RESET = COMMON + r"""
ok(cu.cuInit(0))

def once():
    ctx = P()
    ok(cu.cuDevicePrimaryCtxRetain(ctypes.byref(ctx), 0))
    ok(cu.cuCtxSetCurrent(ctx))
    args = put_all()
    calls(*args, ep.ep_launch(None, None, None, None))
    ok(cu.cuCtxSynchronize())
    return results(args)

want = once()
ok(cu.cuDevicePrimaryCtxReset_v2(0))          # this process's own context
assert all(torch.equal(a, w) for a, w in zip(once(), want))
print("fine")
"""


def passes(program):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", program], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "fine", r.stderr[-2000:]


@pytest.mark.parametrize("captured", ["[False]", "[True]", "[False, True, False]"])
def test_second_context(captured):
    passes(SECOND.replace("CAPTURED", captured))


def test_context_made_again():
    passes(RESET)
