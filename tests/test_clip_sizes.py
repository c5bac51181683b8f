"""The workspace query of lora_clip_gradients answers for the sizes that the call takes,
and no others (host only)."""
import ctypes
import os
import sys

sys.path.insert(0, os.path.dirname(__file__))
from test_linear import lib  # noqa: E402


def test_query_refuses_what_the_call_refuses():
    sgl = lib()
    n, groups = 65536, 1023                        # 67 million parts, more than a launch has workgroups

    def both(n, groups, size):
        sizes, types = (ctypes.c_int64 * n)(*[size] * n), (ctypes.c_int * n)(*[1] * n)
        nbytes = sgl.lib.lora_clip_gradients_workspace_bytes(sizes, types, n, groups)
        at = (ctypes.c_void_p * n)(*[0x10000 + 4 * size * i for i in range(n)])
        # (a workspace of no bytes: no call gets as far as a launch)
        return nbytes, sgl.lib.lora_clip_gradients(at, at, sizes, types, n, groups, 1.0, 0x100, 0x200, 0, None)
    assert both(n, groups, groups) == (0, sgl.LORA_ERR_SHAPE)
    nbytes, st = both(n, 128, 128)                 # 2^23 parts: the most
    assert nbytes >= 8 << 23 and st == sgl.LORA_ERR_BUFFER
    nbytes, st = both(1, 1, 0)
    assert nbytes > 0 and st == sgl.LORA_ERR_BUFFER
