"""A Python function on a stream (a host callback) runs while calls are being made:
the calls let go of the interpreter's lock when they may wait for the GPU."""
import ctypes
import glob
import os

import pytest

from .test_decode_paged import _fa, make

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _runtime():
    for name in ("libcudart.so.13", "libcudart.so"):
        try:
            return ctypes.CDLL(name)
        except OSError:
            pass
    for path in glob.glob(os.path.join(os.path.dirname(torch.__file__), "lib", "libcudart*")):
        return ctypes.CDLL(path)
    pytest.skip("no CUDA runtime to queue a host function with")


def test_a_host_function_runs_while_the_launch_queue_is_full():
    """More calls than a stream's queue holds, behind a function that needs the
    interpreter: a launch then waits for room, which only the function makes."""
    fa = _fa()
    runtime = _runtime()
    kind = ctypes.CFUNCTYPE(None, ctypes.c_void_p)
    x = make([40, 7, 33], 4, 2, 64, 16, seed=3)
    freq = fa.rotary_inv_freq(64, device="cuda")[0]
    pos = torch.arange(3, dtype=torch.int32, device="cuda")
    out, table = torch.empty_like(x["q"]), x["table"].clone()
    k = x["q"][:, :2].contiguous()
    maps = fa.page_maps(x["lens"], pos, table, pos, 16, 9)
    want = fa.rotary(x["q"], pos, freq)
    calls = [lambda: fa.rotary(x["q"], pos, freq, out=out),
             lambda: fa.cache_append(x["q"], k, k, pos, pos, freq, x["k"], x["v"], q_out=out),
             lambda: fa.page_maps(x["lens"], pos, table, pos, 16, 9, out=maps),
             lambda: fa.attention_decode_paged(x["q"], x["k"], x["v"], x["table"], x["lens"])]
    torch.cuda.synchronize()
    for call in calls:
        ran = []
        f = kind(lambda _: ran.append(sum(range(1000))))
        torch.cuda._sleep(20000000)                        # (the queue fills behind this)
        stream = torch.cuda.current_stream().cuda_stream
        assert runtime.cudaLaunchHostFunc(ctypes.c_void_p(stream), f, None) == 0
        for _ in range(3000):
            call()
        torch.cuda.synchronize()
        assert ran == [sum(range(1000))]
    assert torch.equal(fa.rotary(x["q"], pos, freq), want)
