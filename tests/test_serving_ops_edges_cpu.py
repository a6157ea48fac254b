"""The 8-bit cache's dtype beside the calls that do not take it, on the CPU."""
import ctypes
from types import SimpleNamespace

import numpy as np
import pytest

import paged_kv_cache_113_gb300 as pk


@pytest.fixture(scope="module")
def L():
    pk.build()
    return pk.lib()


def test_binding_takes_float8_pools_where_they_serve(L):
    """Calls of fp32 and bf16 pools raise TypeError for a float8 pool, as for any other type, before
    anything else; a descriptor can be had of one."""
    torch = pytest.importorskip("torch")
    kc = torch.zeros((4, 16, 2, 64), dtype=torch.float8_e4m3fn)
    x = torch.zeros((1, 2, 64), dtype=torch.float8_e4m3fn)
    i64, tb, ln = torch.zeros(1, dtype=torch.int64), torch.zeros((1, 4), dtype=torch.int32), torch.ones(1).int()
    items, pairs = torch.zeros((1, 2), dtype=torch.int32), torch.zeros((1, 2), dtype=torch.int64)
    calls = {
        "scatter": lambda c: pk.pk_reshape_and_cache(x, x, i64, c, c),
        "append": lambda c: pk.pk_reshape_and_cache_append(x, x, i64, c, c, tb, ln),
        "copy": lambda c: pk.pk_copy_blocks(c, c, pairs),
        "swap": lambda c: pk.pk_swap_blocks(c, c, c, c, pairs, 0),
        "decode": lambda c: pk.pk_paged_attention_decode(x, x, c, c, tb, ln, 0.1, 64),
        "decode append": lambda c: pk.pk_paged_attention_decode_append(x, x, x, x, i64, c, c, tb, ln, 0.1, 64, 0,
                                                                       items),
        "decode advance": lambda c: pk.pk_paged_attention_decode_advance(x, x, x, x, i64, c, c, tb, ln, ln, 0.1, 64, 0,
                                                                         items),
        "static": lambda c: pk.pk_paged_attention_decode_static(x, x, c, c, tb, ln, 0.1, 64),
        "cascade": lambda c: pk.pk_cascade_attention_decode(x, x, c, c, tb, ln, 0.1, 64, {}),
        "step": lambda c: pk.DecodeStepper(pk.BlockManager(4, 16), [0], 2, 0.1, 4, c, c),
    }
    for name, call in calls.items():
        for pool in (kc, kc.half()):
            with pytest.raises(TypeError, match="float32 or bfloat16"):
                call(pool)
    assert pk.cache_desc(kc).dtype == pk.PK_E4M3
    with pytest.raises(TypeError):
        pk.cache_desc(kc.half())


def test_every_call_of_fp32_and_bf16_pools_refuses_8_bit_ones(L):
    buf = np.zeros(1 << 16, np.uint8)
    p = (buf.ctypes.data + 255) // 256 * 256
    d = pk.CacheDesc(64, 16, 8, 128, pk.PK_E4M3)
    ref, uns = ctypes.byref(d), pk.PK_ERR_UNSUPPORTED
    assert L.pk_reshape_and_cache_append(p, p, p, 1, p, p, ref, p, 4, p, None) == uns
    assert L.pk_swap_blocks(p, p, p, p, 4, p, 1, 0, ref, None) == uns
    assert L.pk_paged_attention_decode(p, p, p, p, p, p, 0.1, 16, 4, 8, 4, 64, 0, None, 0, ref, None) == uns
    assert L.pk_paged_attention_decode_items(p, p, p, p, p, p, 0.1, 4, 8, 4, 64, 0, p, 1, None, 0, ref, 0, None) == uns
    assert L.pk_paged_attention_decode_append(p, p, p, p, p, p, p, p, p, 0.1, 4, 8, 4, 64, 0, p, 1, None, 0, ref,
                                              None) == uns
    assert L.pk_paged_attention_decode_advance(p, p, p, p, p, p, p, p, p, p + 256, 0.1, 4, 8, 4, 64, 0, p, 1, None, 0,
                                               ref, None) == uns
    assert L.pk_cascade_attention_decode(p, p, p, p, p, p, 0.1, 4, 8, 4, 64, 0, p, p, p, p, 1, 2, 16, None, p, 1 << 16,
                                         ref, None) == uns
    assert L.pk_cascade_workspace_size(4, 8, 64, 1, 16, 16, ref) == 0
    steps = pk.StepBuffers()
    steps.meta_host = p
    bm = pk.BlockManager(64, 16)
    ids = np.zeros(1, np.int64)
    assert L.pk_decode_step_prepare(bm._h, ids.ctypes.data, 1, 8, 4, 0, ref, ctypes.byref(steps)) == uns
    assert L.pk_decode_step_launch(1, 8, 0.1, 4, p, p, ref, ctypes.byref(steps), None) in (uns, pk.PK_ERR_INVALID_ARG)


def test_stream_handles_without_the_short_way():
    """A PyTorch without the undocumented lookup serves through the documented one."""
    cuda = SimpleNamespace(current_stream=lambda dev: SimpleNamespace(cuda_stream=1000 + dev))
    assert pk._raw_stream(SimpleNamespace(_C=SimpleNamespace(), cuda=cuda))(3) == 1003
    short = SimpleNamespace(_cuda_getCurrentRawStream=lambda dev: 7 + dev)
    assert pk._raw_stream(SimpleNamespace(_C=short, cuda=cuda))(3) == 10
