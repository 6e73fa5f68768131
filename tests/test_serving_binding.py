"""Host-side checks of the compiled binding of the serving calls: frequencies.  No GPU: every
call is refused, or is an empty call, before anything is enqueued."""
import pytest
import torch

FAKE = 1 << 20  # never dereferenced


@pytest.fixture(scope="module")
def C():
    from kv_cache_eviction_lse_gb300 import build
    build.build()
    from kv_cache_eviction_lse_gb300 import capi
    return capi


def calls(C, f):
    dm = C.dims(1, 2, 1, 64)
    yield lambda: C.kvs_rope(dm, 0, None, 64, f, False, None, None, None, None, stream=0)
    yield lambda: C.kvs_append_paged(dm, 0, 0, None, None, 64, f, False, None, None, None, None, 16,
                                     None, None, 0, None, None, None, 1, None, None, None, 0, stream=0)


def test_frequencies_off_the_host_are_refused(C):
    """Reading them one by one would wait for the device each time and cannot be captured."""
    for dtype in (torch.float64, torch.float32):
        for call in calls(C, torch.zeros(32, dtype=dtype, device="meta")):
            with pytest.raises(ValueError, match="inv_freq must be in host memory"):
                call()


def test_frequencies_of_other_types(C):
    """CPU tensors of any real type and layout; the library refuses a value that is not finite,
    so that it shows which ones were read."""
    for dtype in (torch.float64, torch.float32, torch.float16, torch.bfloat16):
        good = torch.linspace(1, 0.01, 32).to(dtype)
        bad = good.clone()
        bad[31] = float("inf")
        behind = torch.cat([good, bad[31:]])               # what is not needed is not read
        twice = torch.stack([good, bad], 1)[:, 0]          # nor what lies between
        for f in (good, behind, twice, good.clone().requires_grad_()):
            for call in calls(C, f):
                call()
        for f in (bad, torch.stack([good, bad], 1)[:, 1], bad.clone().requires_grad_()):
            for call in calls(C, f):
                with pytest.raises(C.KvsError, match=r"inv_freq\[31\] is not finite"):
                    call()
        for call in calls(C, good[:31]):
            with pytest.raises(ValueError, match="31 frequencies, 32 needed"):
                call()
    for call in calls(C, torch.ones(32, dtype=torch.int64)):
        call()
    for call in calls(C, torch.ones(32, dtype=torch.complex64)):
        with pytest.raises(TypeError):
            call()
