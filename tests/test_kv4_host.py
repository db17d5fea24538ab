"""CPU checks of the 4-bit cache: the definition's own properties, and what the entry points refuse on
the host before anything is launched."""
import ctypes

import pytest
import torch

import kv4_ref as ref


@pytest.fixture(scope="module")
def lib():
    from eagle_speculative_decoding_draft_gb300 import build, _lib
    build.build()
    return _lib.load()


def cache(**kw):
    from eagle_speculative_decoding_draft_gb300._lib import KV4CacheStruct
    f = dict(kv_heads=2, head_dim=64, page_size=32, num_pages=10, max_pages=4, pages=256, table=256, lengths=256)
    f.update(kw)
    return KV4CacheStruct(*(f[k] for k, _ in KV4CacheStruct._fields_))


BAD = [dict(kv_heads=0), dict(kv_heads=1025), dict(head_dim=48), dict(head_dim=0), dict(head_dim=160), dict(page_size=8),
       dict(page_size=48), dict(page_size=2048), dict(num_pages=0), dict(max_pages=0), dict(max_pages=1 << 27),
       dict(page_size=1024, max_pages=(1 << 20) + 1)]
BAD_POINTERS = [dict(pages=None), dict(table=None), dict(lengths=None), dict(pages=264), dict(table=258)]
P = ctypes.c_void_p


def test_pool_bytes(lib):
    """640 bytes for 16 tokens of 32 dims: 4 bits a value and 4 bytes a group, keys and values."""
    for kw in (dict(), dict(head_dim=128, page_size=16), dict(head_dim=96, kv_heads=3), dict(head_dim=32, page_size=1024, num_pages=7)):
        c = cache(pages=None, table=None, lengths=None, **kw)
        assert lib.eagle_kv4_pages_bytes(ctypes.byref(c)) == \
            c.num_pages * c.page_size * c.kv_heads * 2 * (c.head_dim // 2 + c.head_dim // 8)
    big = cache(head_dim=128, kv_heads=32, page_size=1024, num_pages=1 << 20)
    assert lib.eagle_kv4_pages_bytes(ctypes.byref(big)) == (1 << 20) * 1024 * 32 * 160
    for bad in BAD:
        assert lib.eagle_kv4_pages_bytes(ctypes.byref(cache(**bad))) == 0
    assert lib.eagle_kv4_pages_bytes(None) == 0


def append(lib, c, batch=2, src_rows=5, slots=5, k=P(256), v=P(256), ld=128, select=None, count=None, start=None):
    return lib.eagle_kv4_append(ctypes.byref(c), batch, src_rows, slots, k, v, ld, select, count, start, None, None)


def read(lib, c, batch=2, rows=5, start=None, k=P(256), v=P(256), dtype=0):
    return lib.eagle_kv4_read(ctypes.byref(c), batch, rows, start, k, v, dtype, None, None)


def attend(lib, c, batch=2, nodes=3, heads=4, q=P(256), ldq=256, k=P(256), v=P(256), ldkv=128, mask=None, out=P(256),
           ws=P(256), nbytes=1 << 40):
    return lib.eagle_kv4_attention(ctypes.byref(c), batch, nodes, heads, q, ldq, k, v, ldkv, mask, out, ws, nbytes, None, None)


@pytest.mark.parametrize("bad", BAD + BAD_POINTERS, ids=str)
def test_every_call_refuses_an_unusable_cache(lib, bad):
    c = cache(**bad)
    assert append(lib, c) == 1 and read(lib, c) == 1 and attend(lib, c) == 1
    assert lib.eagle_kv4_attention_workspace_bytes(ctypes.byref(c), 3, 4) == 0


@pytest.mark.parametrize("kw", [dict(batch=-1), dict(src_rows=-1), dict(slots=-1), dict(slots=6), dict(k=None), dict(v=None),
                                dict(k=P(264)), dict(v=P(258)), dict(ld=120), dict(ld=132), dict(select=P(257)),
                                dict(count=P(258)), dict(start=P(1))], ids=str)
def test_append_refuses(lib, kw):
    assert append(lib, cache(), **kw) == 1


@pytest.mark.parametrize("kw", [dict(batch=-1), dict(rows=-1), dict(dtype=2), dict(k=None), dict(v=None), dict(k=P(264)),
                                dict(start=P(2))], ids=str)
def test_read_refuses(lib, kw):
    assert read(lib, cache(), **kw) == 1


@pytest.mark.parametrize("kw", [dict(batch=-1), dict(nodes=0), dict(nodes=4098), dict(heads=0), dict(heads=3), dict(heads=65538),
                                dict(q=None), dict(out=None), dict(ws=None), dict(k=None), dict(v=None), dict(ldq=248),
                                dict(ldq=260), dict(ldkv=120), dict(ldkv=132), dict(q=P(264)), dict(k=P(264)), dict(out=P(8)),
                                dict(ws=P(128)), dict(mask=P(258)), dict(k=None, v=None, mask=P(256)),
                                dict(nodes=4097, heads=65536)], ids=str)
def test_attention_refuses(lib, kw):
    assert attend(lib, cache(), **kw) == 1


@pytest.mark.parametrize("limit,tile", [(0, 0), (-1, 0), (10 ** 10 + 1, 0), (1000, -1)])
def test_stall_hook_refuses(lib, limit, tile):
    c = cache()
    call = lambda cache_ref, limit, tile: lib.eagle_test_kv4_stall(cache_ref, 2, 3, 4, P(256), P(256), P(256), None, P(256), P(256), 1 << 40,
                                                                   limit, tile, None, None)
    assert call(ctypes.byref(c), limit, tile) == 1
    assert call(None, 1000, 0) == 1 and call(ctypes.byref(cache(page_size=24)), 1000, 0) == 1


def test_empty_batches_do_nothing(lib):
    c = cache()
    assert append(lib, c, batch=0, k=None, v=None) == 0
    assert read(lib, c, batch=0, k=None, v=None) == 0
    assert read(lib, c, rows=0, k=None, v=None) == 0
    assert attend(lib, c, batch=0, q=None, k=None, v=None, out=None, ws=None) == 0


def test_decoder_layer_refuses(lib):
    from eagle_speculative_decoding_draft_gb300._lib import DecoderLayerWeights
    f = dict(hidden=256, heads=4, kv_heads=2, head_dim=64, inter=512, rope_theta=1e4, rms_eps=1e-6,
             w_qkv=256, w_o=256, w_norm=256, w_gu=256, w_d=256)

    def call(c, nodes=9, x=P(256), ws=P(256), **kw):
        w = DecoderLayerWeights(*({**f, **kw}[k] for k, _ in DecoderLayerWeights._fields_))
        if lib.eagle_decoder_layer_kv4_workspace_bytes(ctypes.byref(w), ctypes.byref(c), 2, nodes) != 0:
            return None  # there is a device: the sizes pass
        return lib.eagle_decoder_layer_kv4(ctypes.byref(w), ctypes.byref(c), 2, nodes, x, P(256), None, P(256), None, None, ws,
                                           1 << 40, None, None)

    for bad in (dict(kv_heads=4), dict(head_dim=128), dict(page_size=24), dict(pages=None)):
        assert call(cache(**bad)) == 1
    assert call(cache(), nodes=0) == 1 and call(cache(), nodes=4098) == 1
    assert call(cache(), heads=3) == 1 and call(cache(), rope_theta=0.0) == 1


class Elsewhere:
    """Looks like a contiguous CUDA tensor; no kernel may get its address."""

    def __init__(self, shape, dtype, index=0):
        self.shape, self.dtype, self.device, self.is_cuda = shape, dtype, torch.device("cuda", index), True

    def is_contiguous(self):
        return True

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n

    def data_ptr(self):
        raise AssertionError("the call went on with it")


@pytest.mark.parametrize("which", ["positions", "mask", "out", "workspace"])
def test_decoder_layer_over_the_cache_refuses_tensors_on_another_device(lib, which):
    import contextlib
    import types
    from eagle_speculative_decoding_draft_gb300.engine import DecoderLayer
    lay = DecoderLayer.__new__(DecoderLayer)
    lay.hidden, lay.heads, lay.kv_heads, lay.head_dim, lay.device = 256, 4, 2, 64, torch.device("cuda", 0)
    lay.w = ctypes.c_int(0)
    lay._lib = types.SimpleNamespace(eagle_decoder_layer_kv4_workspace_bytes=lambda *a: 1024)
    kv = types.SimpleNamespace(batch=2, device=torch.device("cuda", 0), _on=lambda stream: contextlib.nullcontext(), _ref=None)
    on = lambda name: 1 if name == which else 0
    args = dict(positions=Elsewhere((2, 9), torch.int32, on("positions")), mask=Elsewhere((2, 9, 1), torch.int32, on("mask")),
                out=Elsewhere((2, 9, 256), torch.bfloat16, on("out")), workspace=Elsewhere((1024,), torch.uint8, on("workspace")))
    with pytest.raises(ValueError, match=f"{which} is on cuda:1"):
        lay.kv4(Elsewhere((2, 9, 256), torch.bfloat16), kv, **args)


def test_a_stream_of_another_device_is_refused():
    import types
    from eagle_speculative_decoding_draft_gb300.engine import DecoderLayer
    from eagle_speculative_decoding_draft_gb300.kv4 import KV4Cache
    c = KV4Cache.__new__(KV4Cache)
    c.device, c._index, c.batch, c._tail, c._lib, c._ref = torch.device("cuda", 0), 0, 2, (2, 64), None, None
    lay = DecoderLayer.__new__(DecoderLayer)
    lay.hidden, lay.device = 256, c.device
    stream = types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0)
    x = Elsewhere((2, 9, 256), torch.bfloat16)
    for call in (lambda: c.status(stream=stream), lambda: c.read(rows=3, stream=stream),
                 lambda: lay.kv4(x, c, Elsewhere((2, 9), torch.int32), stream=stream)):
        with pytest.raises(ValueError, match="stream is on cuda:1"):
            call()


@pytest.mark.parametrize("scale", [1.0, 1e-4, 300.0])
def test_the_definition_holds_its_error_bound(scale):
    """No value is further than half a step from what its code stands for (no code is clamped), and
    the step is at most the range / 15 and its fp16 roundings."""
    g = torch.Generator().manual_seed(0)
    x = (scale * (torch.randn(500, 128, generator=g) + torch.randn(128, generator=g))).to(torch.bfloat16)
    m, s, c = ref.parts(x)
    err = (m + s * c - x.double().unflatten(-1, (-1, 32))).abs()
    assert torch.all(err <= s / 2 * (1 + 1e-12))
    assert torch.all(c == c.round()) and c.min() == 0 and c.max() == 15
    span = (x.double().unflatten(-1, (-1, 32)).amax(-1, keepdim=True) - m)
    assert torch.all(s <= span / 15 * (1 + 2.0 ** -10) + 2.0 ** -24)


def test_attention_reference_against_a_plain_loop():
    """The reference the GPU tests use, against a loop over rows and keys on small sizes."""
    import math
    g = torch.Generator().manual_seed(1)
    n, H, Hk, D, t = 3, 4, 2, 32, 5
    r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)
    q, kc, vc, kn, vn = r(n, H, D), r(t, Hk, D), r(t, Hk, D), r(n, Hk, D), r(n, Hk, D)
    see = ref.sees(n, t, None, "cpu")
    o, tol = ref.attend(q, kc, vc, kn, vn, see)
    k = torch.cat([ref.stands_for(kc), kn.double()])
    v = torch.cat([ref.stands_for(vc), vn.double()])
    for i in range(n):
        for h in range(H):
            w = [math.exp(float(q[i, h].double() @ k[j, h // 2]) / math.sqrt(D)) if see[i, j] else 0.0 for j in range(t + n)]
            want = sum(a * v[j, h // 2] for j, a in enumerate(w)) / sum(w)
            assert torch.allclose(o[i, h], want, rtol=1e-12, atol=1e-12)
    assert torch.all(tol > 0) and float(tol.max()) < 0.05
