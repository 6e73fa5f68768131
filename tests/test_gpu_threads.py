"""Calls of the surrogate from host threads whose models differ in hidden size."""
import ctypes
import threading

import pytest
import torch

from .gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def C():
    need_gpu()
    from kv_cache_eviction_lse_gb300 import build
    build.build()
    from kv_cache_eviction_lse_gb300 import capi
    return capi


@pytest.mark.parametrize("Hkv, sizes", [(8, (12800, 4096)), (16, (6400, 4096))])
def test_threads_with_hidden_sizes_of_their_own(C, Hkv, sizes):
    """Blocks of 64 to 200 KB of shared memory, launched in turn by all."""
    T = 4900  # enough tokens for the kernel whose blocks keep a head group's weights

    class Model:
        def __init__(self, Dh, seed):
            gen = torch.Generator(device="cuda").manual_seed(seed)
            self.dm = C.dims(1, Hkv, Hkv, 128, Dh)
            self.h = torch.randn(1, T, Dh, generator=gen, device="cuda").to(torch.bfloat16)
            self.W = (torch.randn(1, Dh, Hkv, generator=gen, device="cuda") / Dh ** 0.5).to(torch.bfloat16)
            self.b = torch.randn(1, Hkv, generator=gen, device="cuda")
            self.z = torch.empty(1, Hkv, T, device="cuda")
            self.stream, self.raised = torch.cuda.Stream(), []
            # the C function itself: the less Python between two calls, the likelier they meet
            p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
            self.args = (ctypes.byref(self.dm), p(self.h), T, p(self.W), p(self.b), p(self.z), 0.0, 0, None, None,
                         ctypes.c_void_p(self.stream.cuda_stream))
            torch.cuda.synchronize()
            assert C._lib.kvs_surrogate(*self.args) == C.KVS_OK
            torch.cuda.synchronize()
            self.alone = self.z.clone()

        def work(self):
            for i in range(20000):
                st = C._lib.kvs_surrogate(*self.args)
                if st != C.KVS_OK:
                    self.raised.append((i, st))
                if i % 200 == 199:
                    self.stream.synchronize()

    models = [Model(Dh, i) for i, Dh in enumerate(sizes * 2)]
    torch.cuda.synchronize()
    threads = [threading.Thread(target=m.work) for m in models]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not any(m.raised for m in models), [m.raised[:3] for m in models]
    assert C.kvs_device_error() == 0
    for m in models:
        assert torch.equal(m.z, m.alone)
