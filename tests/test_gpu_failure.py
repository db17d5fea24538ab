"""Failure detection without a GPU fault: a device wait that nothing will satisfy gives up after
its limit, the kernel reports EAGLE_ERR_DEVICE_TIMEOUT through the status word and returns, and
the context stays usable (a GEMM launched afterwards is still correct and deterministic)."""
import ctypes
import time

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available()
    return torch.device("cuda", 0)


def test_bounded_wait_times_out_and_the_context_survives(dev):
    from eagle_speculative_decoding_draft_gb300 import _lib
    from eagle_speculative_decoding_draft_gb300.engine import linear_bf16
    lib = _lib.load()
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    for limit_ns in (1_000, 1_000_000, 20_000_000):
        t0 = time.perf_counter()
        rc = lib.eagle_test_bounded_wait(limit_ns, ctypes.c_void_p(status.data_ptr()), st)
        dt = time.perf_counter() - t0
        assert rc == 5, rc  # EAGLE_ERR_DEVICE_TIMEOUT
        assert dt >= limit_ns * 1e-9 * 0.5
        assert int(status.item()) == 0  # read and cleared
    # the context is intact: a GEMM afterwards matches a float64 reference
    rng = np.random.default_rng(0)
    W = torch.from_numpy((rng.standard_normal((300, 640)) * 0.05).astype(np.float32)).to(torch.bfloat16)
    X = torch.from_numpy(rng.standard_normal((7, 640)).astype(np.float32)).to(torch.bfloat16)
    y = linear_bf16(W.to(dev), X.to(dev)).cpu().double()
    ref = X.double() @ W.double().T
    assert torch.allclose(y, ref, atol=1e-3, rtol=1e-3)


def test_bounded_wait_rejects_bad_arguments(dev):
    from eagle_speculative_decoding_draft_gb300 import _lib
    lib = _lib.load()
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    P = ctypes.c_void_p
    assert lib.eagle_test_bounded_wait(0, P(status.data_ptr()), None) == 1
    assert lib.eagle_test_bounded_wait(10**11, P(status.data_ptr()), None) == 1
    assert lib.eagle_test_bounded_wait(1000, None, None) == 1


@pytest.mark.parametrize("B,n,H,Hk,D,cached,tile", [
    (3, 1, 4, 4, 128, 900, 0), (40, 8, 8, 8, 64, 200, 3),              # few query rows
    (400, 200, 1, 1, 128, 130, 0), (400, 150, 1, 1, 128, 260, 2),      # a stream a half of the rows
    (400, 70, 1, 1, 64, 130, 1), (2, 65, 8, 2, 96, 1000, 0),           # both streams on the same rows; one tile a CTA
], ids=lambda v: str(v))
def test_kv4_attention_gives_up_when_its_copies_stop(dev, B, n, H, Hk, D, cached, tile):
    """Each CTA's copying warp stops at one of its tiles, so that every other warp's waits run out.  Some tiles
    of new values hold a NaN (whose rows take barriers of their own) and others none.  The call ends, reports the
    timeout, and the next one is right."""
    from eagle_speculative_decoding_draft_gb300 import KV4Cache, _lib
    pages = -(-cached // 32)
    c = KV4Cache(B, Hk, D, num_pages=B * pages, max_pages=pages, page_size=32)
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
    c.append(r(B, cached, Hk, D), r(B, cached, Hk, D))
    q, k, v = r(B, n, H, D), r(B, n, Hk, D), r(B, n, Hk, D)
    v[::2, n // 2, :, 1] = float("nan")
    v[1::3, n - 1, :, 2] = float("inf")
    want = c.attention(q, k, v)
    c.status()
    out = torch.empty_like(q)
    nbytes = c.attention_workspace_bytes(n, H)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    P = ctypes.c_void_p
    for _ in range(2):
        t0 = time.perf_counter()
        assert c._lib.eagle_test_kv4_stall(c._ref, B, n, H, P(q.data_ptr()), P(k.data_ptr()), P(v.data_ptr()), None, P(out.data_ptr()),
                                           P(ws.data_ptr()), nbytes, 20_000_000, tile, P(c._status.data_ptr()),
                                           P(torch.cuda.current_stream().cuda_stream)) == 0
        with pytest.raises(_lib.EagleError, match="TIMEOUT"):
            c.status()
        assert 0.01 < time.perf_counter() - t0 < 5
    got = c.attention(q, k, v)
    c.status()
    assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want)) and torch.equal(got.isnan(), want.isnan())
