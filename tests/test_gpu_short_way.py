"""GPU tests of the extension module _calls beside other threads: it lets go of the interpreter's lock for
the time in which it allocates outputs and is in the library."""
import ctypes
import threading

import pytest
import torch

from gpu_util import say

pytestmark = pytest.mark.gpu

ENTRIES = ("sparse_ffn_rms_norm", "sparse_ffn_quantize_mx4", "sparse_ffn_dequantize_mx4",
           "sparse_ffn_mx4_matmul_work_bytes", "sparse_ffn_mx4_matmul")


@pytest.fixture(scope="module", autouse=True)
def P():
    import activation_sparse_decode_rank_amd as P  # fails loudly without the HIP library
    torch.cuda.init()
    yield P


def calls(P):
    """A regular call of every operator."""
    x = torch.randn((6, 128), device="cuda")
    q, s = P.quantize_mx4(x)
    return [lambda: P.rms_norm(x), lambda: P.rms_norm(x, residual=x, out="i8"),
            lambda: P.rms_norm(x, residual=x, out="mx4"), lambda: P.quantize_mx4(x),
            lambda: P.dequantize_mx4(q, s), lambda: P.mx4_matmul(x, q, s),
            lambda: P.mx4_matmul(q, q, s, x_scale=s)]


def test_the_lock_is_free_inside_the_library(P):
    """In the place of the library's entry points the interpreter's own question whether this thread holds
    the lock: 0 is the library's status for success, 1 would be raised as an error."""
    from activation_sparse_decode_rank_amd import _calls
    say("lock in the library")
    held = ctypes.cast(ctypes.pythonapi.PyGILState_Check, ctypes.c_void_p).value
    todo = calls(P)
    try:
        _calls.bind(*[held] * len(ENTRIES))
        for call in todo:
            call()
    finally:
        _calls.bind(*(P._native.address(e) for e in ENTRIES))
    want = [c() for c in todo]
    assert all(torch.isfinite(t.float()).all() for w in want for t in (w if isinstance(w, tuple) else (w,)))


def test_calls_of_many_threads(P):
    """The same calls from several threads at once, each on a stream of its own: the same bits."""
    say("threads")
    todo = calls(P)
    want = [c() for c in todo]
    torch.cuda.synchronize()
    wrong = []

    def work():
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(200):
                for c, w in zip(todo, want):
                    got = c()
                    for a, b in zip(*((t if isinstance(t, tuple) else (t,)) for t in (got, w))):
                        if not torch.equal(a, b):
                            wrong.append(c)
            stream.synchronize()

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
