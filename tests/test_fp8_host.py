"""CPU checks of the 8-bit operators: what the entry points refuse on the host before anything is launched."""
import ctypes

import pytest

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    from eagle_speculative_decoding_draft_gb300 import build, _lib
    build.build()
    return _lib.load()


def quantize(lib, x=P(256), ldx=64, rows=4, cols=64, y=P(256), ldy=64, scale=P(256)):
    return lib.eagle_quantize_rows(x, ldx, rows, cols, y, ldy, scale, None)


def norm(lib, x=P(256), ldx=64, res=P(256), ldr=64, w=P(256), eps=1e-5, rows=4, cols=64, s=P(256), lds=64, dtype=2, y=P(256),
         ldy=64, scale=P(256)):
    return lib.eagle_rms_norm(x, ldx, res, ldr, w, eps, rows, cols, s, lds, dtype, y, ldy, scale, None)


@pytest.mark.parametrize("bad", [dict(x=None), dict(y=None), dict(scale=None), dict(x=P(264)), dict(y=P(264)), dict(scale=P(258)),
                                 dict(ldx=63), dict(ldx=68), dict(ldy=72), dict(ldy=48), dict(rows=-1), dict(cols=0)], ids=str)
def test_quantize_rows_refuses(lib, bad):
    assert quantize(lib, **bad) == 1


@pytest.mark.parametrize("bad", [dict(x=None), dict(w=None), dict(y=None), dict(scale=None), dict(x=P(264)), dict(res=P(264)),
                                 dict(w=P(260)), dict(s=P(264)), dict(y=P(264)), dict(scale=P(257)), dict(ldx=60), dict(ldx=68),
                                 dict(ldr=56), dict(ldr=65), dict(lds=56), dict(lds=65), dict(ldy=72), dict(rows=-1), dict(cols=0),
                                 dict(eps=-1.0), dict(eps=float("nan")), dict(dtype=0), dict(dtype=3), dict(dtype=1),
                                 dict(res=None)], ids=str)
def test_rms_norm_refuses(lib, bad):
    assert norm(lib, **bad) == 1


def test_rows_limits(lib):
    assert quantize(lib, cols=32769, ldx=32776, ldy=32784) == 2
    assert norm(lib, cols=32769, ldx=32776, ldr=32776, lds=32776, ldy=32784) == 2
    assert quantize(lib, rows=0, x=None, y=None, scale=None) == 0
    assert norm(lib, rows=0) == 0


def linear(lib, ws=P(256), nbytes=1 << 40, status=None, **kw):
    from eagle_speculative_decoding_draft_gb300._lib import LinearArgs
    f = dict(rows=20, out_features=64, in_features=128, dtype=2, y_dtype=1, act=0, w=256, x=256, ldw=128, ldx=128, w_scale=256,
             x_scale=256, bias=256, residual=256, ldr=64, y=256, ldy=64)
    f.update(kw)
    return lib.eagle_linear(ctypes.byref(LinearArgs(*(f[k] for k, _ in LinearArgs._fields_))), ws, nbytes, status, None)


@pytest.mark.parametrize("bad", [dict(rows=-1), dict(rows=32769), dict(out_features=0), dict(in_features=0), dict(dtype=0), dict(dtype=3),
                                 dict(y_dtype=2), dict(act=-1), dict(act=4), dict(w=None), dict(x=None), dict(y=None), dict(nbytes=4095),
                                 dict(w=264), dict(x=264), dict(w_scale=None), dict(x_scale=None), dict(w_scale=258), dict(x_scale=258),
                                 dict(bias=257), dict(residual=257), dict(y=257), dict(ws=P(128)), dict(status=P(258)), dict(ldw=112),
                                 dict(ldx=136), dict(ldw=136), dict(ldy=63), dict(ldr=63), dict(dtype=1), dict(y_dtype=0, y=258),
                                 dict(dtype=1, w_scale=None, x_scale=None, ldw=132), dict(out_features=(1 << 28) + 1, ldy=1 << 30, residual=None),
                                 dict(in_features=(1 << 28) + 1, ldw=1 << 30, ldx=1 << 30)],
                         ids=str)
def test_linear_refuses(lib, bad):
    assert linear(lib, **bad) == 1


def test_linear_edges(lib):
    assert linear(lib, rows=0, w=None, x=None, y=None, ws=None) == 0
    assert lib.eagle_linear(None, P(256), 1 << 30, None, None) == 1
    assert lib.eagle_linear_epilogue_workspace_bytes(0) == 0 and lib.eagle_linear_epilogue_workspace_bytes(32769) == 0


def rotary(lib, batch=2, src_rows=5, slots=5, k=P(256), v=P(256), ld=128, positions=None, theta=1e4, heads=4, q=P(256), ldq=256, out=P(256),
           select=None, count=None, start=None, **kw):
    from test_kv4_host import cache
    return lib.eagle_kv4_append_rotary(ctypes.byref(cache(**kw)), batch, src_rows, slots, k, v, ld, positions, theta, heads, q, ldq, out,
                                       select, count, start, None, None)


@pytest.mark.parametrize("bad", [dict(head_dim=48), dict(pages=None), dict(batch=-1), dict(src_rows=-1), dict(slots=-1), dict(slots=6),
                                 dict(k=None), dict(v=None), dict(ld=120), dict(ld=132), dict(k=P(264)), dict(v=P(264)), dict(theta=0.0),
                                 dict(theta=-1.0), dict(theta=float("nan")), dict(select=P(256)), dict(positions=P(258)), dict(out=None),
                                 dict(q=None), dict(heads=0), dict(heads=65537, ldq=1 << 23), dict(ldq=248), dict(ldq=260), dict(q=P(264)),
                                 dict(out=P(264)), dict(count=P(257)), dict(start=P(257))], ids=str)
def test_append_rotary_refuses(lib, bad):
    assert rotary(lib, **bad) == 1


def test_append_rotary_of_no_requests(lib):
    assert rotary(lib, batch=0) == 0


def fp8_layer(lib, batch=2, nodes=3, x=P(256), positions=P(256), mask=P(256), out=P(256), k_new=P(256), v_new=P(256), ws=P(256), nbytes=1 << 40,
              status=None, cache=None, **kw):
    from eagle_speculative_decoding_draft_gb300._lib import DecoderLayerFP8Weights
    from test_kv4_host import cache as make
    f = dict(hidden=64, heads=4, kv_heads=2, head_dim=64, inter=48, rope_theta=1e4, rms_eps=1e-6, w_qkv=256, w_o=256, w_norm=256, w_gu=256,
             w_d=256, s_qkv=256, s_o=256, s_gu=256, s_d=256)
    f.update(kw)
    w = DecoderLayerFP8Weights(*(f[k] for k, _ in DecoderLayerFP8Weights._fields_))
    c = make(**(cache or {}))
    if nbytes is None:
        return lib.eagle_decoder_layer_fp8_kv4_workspace_bytes(ctypes.byref(w), ctypes.byref(c), batch, nodes)
    return lib.eagle_decoder_layer_fp8_kv4(ctypes.byref(w), ctypes.byref(c), batch, nodes, x, positions, mask, out, k_new, v_new, ws, nbytes,
                                           status, None)


@pytest.mark.parametrize("bad", [dict(hidden=72), dict(hidden=0), dict(hidden=32784), dict(inter=40), dict(inter=32784), dict(heads=3),
                                 dict(heads=1024), dict(head_dim=96), dict(kv_heads=4), dict(rope_theta=0.0), dict(rms_eps=-1.0),
                                 dict(w_qkv=None), dict(w_o=None), dict(w_norm=None), dict(w_gu=None), dict(w_d=None), dict(s_qkv=None),
                                 dict(s_o=None), dict(s_gu=None), dict(s_d=None), dict(w_gu=264), dict(s_d=258), dict(batch=-1),
                                 dict(nodes=0), dict(nodes=4098), dict(batch=11, nodes=3000), dict(x=None), dict(positions=None),
                                 dict(out=None), dict(x=P(264)), dict(out=P(264)), dict(k_new=None), dict(v_new=P(264)), dict(ws=None),
                                 dict(ws=P(128)), dict(mask=P(258)), dict(status=P(258)), dict(cache=dict(pages=None))], ids=str)
def test_fp8_layer_refuses(lib, bad):
    assert fp8_layer(lib, **bad) == 1


def test_fp8_layer_edges(lib):
    assert fp8_layer(lib, batch=0, x=None, out=None, ws=None) == 0
    for bad in (dict(batch=0), dict(nodes=0), dict(hidden=72), dict(batch=11, nodes=3000), dict(cache=dict(head_dim=96))):
        assert fp8_layer(lib, nbytes=None, **bad) == 0


def test_status_of_products_without_a_device(lib):
    """The word is the device's: without one there is none to read."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("there is a device")
    assert not lib.eagle_linear_status_word() and lib.eagle_linear_status(None) == 4
