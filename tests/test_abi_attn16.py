"""Host checks of the rotary, 16-bit cache and prompt calls: refused before anything is launched (no GPU needed)."""

import ctypes

import pytest


@pytest.fixture(scope="module")
def L():
    from verify_bs_step_gb300 import _build
    _build.build()
    import verify_bs_step_gb300 as vbs
    return vbs.lib()


def test_rotary(L):
    import verify_bs_step_gb300 as vbs
    out = (ctypes.c_double * 128)()
    good = (64, 10000.0, 0, 1.0, 8192.0, 1.0, 4.0)
    assert L.rope_frequencies(*good, out) == vbs.OK
    for at, bad in ((0, -2), (0, 3), (0, 258), (1, 0.0), (1, float("inf")), (1, float("nan")), (2, 4), (2, -1)):
        args = list(good)
        args[at] = bad
        assert L.rope_frequencies(*args, out) == vbs.EINVAL, (at, bad)
    assert L.rope_frequencies(*good, None) == vbs.EINVAL
    for bad in ((64, 1e4, 1, 0.0, 1, 1, 4), (64, 1e4, 3, 2.0, 0.0, 1, 4), (64, 1e4, 3, 2.0, 10, 4, 4), (2, 1e4, 2, 2.0, 1, 1, 4),
                (64, 1e4, 1, float("nan"), 1, 1, 4)):
        assert L.rope_frequencies(*bad, out) == vbs.EINVAL, bad
    ctx = ctypes.c_void_p()
    for D, rot, layout, amp in ((0, 0, 0, 1.0), (257, 64, 0, 1.0), (64, 66, 0, 1.0), (64, 7, 0, 1.0), (64, -2, 0, 1.0), (64, 64, 2, 1.0),
                                (64, 64, 0, float("inf"))):
        assert L.rope_init(ctypes.byref(ctx), D, rot, layout, out, amp) == vbs.EINVAL and not ctx.value
    assert L.rope_init(ctypes.byref(ctx), 64, 64, 0, None, 1.0) == vbs.EINVAL
    assert L.rope_init(None, 64, 64, 0, out, 1.0) == vbs.EINVAL
    out[3] = float("nan")
    assert L.rope_init(ctypes.byref(ctx), 64, 64, 0, out, 1.0) == vbs.EINVAL
    assert L.rope_apply(None, 1, None, 1, None, 0, 0, None, 0, 0, 1, None, 0, 0, None, 0, 0, 0, None) == vbs.EINVAL
    assert L.rope_destroy(None) == vbs.OK


def test_cache(L):
    import verify_bs_step_gb300 as vbs
    ctx = ctypes.c_void_p()
    assert L.kv16_init(ctypes.byref(ctx), None, 4, 1) == vbs.EINVAL and not ctx.value
    assert L.kv16_init(None, None, 4, 1) == vbs.EINVAL
    assert L.kv16_append(None, 0, 1, None, 1, None, 0, 0, None, 0, 0, None, None, None, 0, 0, None, 0, 0, None, 0, 0) == vbs.EINVAL
    assert L.kv16_plan(None, None, 1) == vbs.EINVAL
    assert L.kv16_attention(None, 0, None, 0, 0, 0, 1.0, None, 0, 0, 0) == vbs.EINVAL
    assert L.kv16_destroy(None) == vbs.OK


def test_prompts(L):
    import verify_bs_step_gb300 as vbs
    ctx = ctypes.c_void_p()
    for heads, kv_heads, D in ((0, 1, 64), (4, 0, 64), (4, 3, 64), (4, 2, 0), (4, 2, 12), (4, 2, 264), (1 << 17, 1, 64)):
        assert L.pattn_init(ctypes.byref(ctx), heads, kv_heads, D, None) == vbs.EINVAL and not ctx.value
    assert L.pattn_init(None, 4, 2, 64, None) == vbs.EINVAL
    assert L.pattn_run(None, 1, 1, None, None, 0, 0, None, 0, 0, None, 0, 0, 1, 1.0, None, 0, 0) == vbs.EINVAL
    n = ctypes.c_int()
    assert L.pattn_kernel(None, ctypes.byref(n)) == vbs.EINVAL and L.pattn_status(None) == vbs.EINVAL
    assert L.pattn_destroy(None) == vbs.OK


@pytest.mark.parametrize("name", ["rope_args", "kv16_args", "kv16_query", "pattn_args"])
def test_structs_of_arguments(L, name):
    """The binding packs them as the header declares them; NULL is refused."""
    import os
    import re
    import struct
    import verify_bs_step_gb300 as vbs
    from verify_bs_step_gb300 import _build
    text = open(os.path.join(_build.INCLUDE, "vbs.h")).read()
    body = re.search(r"typedef struct vbs_%s \{(.*?)\}" % name, text, re.S).group(1)
    code = ""
    for line in body.split(";"):
        kind, names = re.match(r"\s*(const \w+ ?\*|void ?\*|vbs_stream_t|int64_t|int|float)\s*(.*)", line + " ", re.S).groups() if line.strip() else ("", "")
        code += {"int64_t": "q", "int": "i", "float": "f"}.get(kind, "Q" if kind else "") * (names.count(",") + 1 if names.strip() else 0)
    packed = {"rope_args": vbs._ROPE_ARGS, "kv16_args": vbs._KV16_ARGS, "kv16_query": vbs._KV16_QUERY, "pattn_args": vbs._PATTN_ARGS}[name]
    assert len(code) > 9 and packed.format.replace(" ", "") == "@" + code
    assert packed.size == struct.calcsize("@" + code)
    call = {"rope_args": L.rope_apply_args, "kv16_args": L.kv16_append_args, "kv16_query": L.kv16_attention_args,
            "pattn_args": L.pattn_run_args}[name]
    assert call(None, None) == vbs.EINVAL
    assert call(None, packed.pack(*([0] * len(code)))) == vbs.EINVAL
