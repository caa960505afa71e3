"""What the entry points of the cache in 4 or 8 bits refuse, on the host (no GPU: nothing is enqueued)."""
import ctypes

import pytest
import torch

A = 4096  # an aligned address that is never read


@pytest.fixture(scope="module")
def kv():
    import __graft_entry__
    __graft_entry__.build_library()
    from attention_fa_fwd_02_gb300 import kv as m
    return m


def cache(kv, **kw):
    block = 16 * (64 + 8)
    d = dict(K=A, V=A, table=A, lens=A, refs=A, status=A, plane_stride=100 * 2 * block, page_stride=2 * block, head_stride=block,
             table_stride=8, planes=3, num_pages=100, page_size=16, HKV=2, D=128, max_slots=4, max_pages=8, bits=4, group=64, dtype=1)
    d.update(kw)
    return kv.fakv_qcache(**d)


def tokens(kv, **kw):
    d = dict(B=2, T=3, H=4, plane=0, q_token=512, q_head=128, k_token=256, k_head=128, v_token=256, v_head=128, scale=0.1, causal=1,
             window=0, out_dtype=1)
    d.update(kw)
    return kv.fakv_tokens(**d)


def calls(kv, c, p):
    lib = kv._lib()
    C, P = ctypes.byref(c), ctypes.byref(p)
    return (lib.fakv_qattend(A, A, A, A, None, C, P, None), lib.fakv_qappend(A, A, A, A, A, None, None, C, P, None),
            lib.fakv_qread(A, A, A, None, None, C, P, None))


def test_struct_layout_matches_the_header(kv):
    import os
    import subprocess
    import sys
    import tempfile
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    fields = [n for n, _ in kv.fakv_qcache._fields_]
    src = '#include <stddef.h>\n#include <stdio.h>\n#include "fakv.h"\nint main(void) { printf("%zu", sizeof(fakv_qcache));\n' + \
        "".join(f'printf(" %zu", offsetof(fakv_qcache, {n}));\n' for n in fields) + "return 0; }\n"
    with tempfile.TemporaryDirectory() as d:
        with open(f"{d}/x.c", "w") as f:
            f.write(src)
        subprocess.run(["gcc", "-I", os.path.join(root, "include"), f"{d}/x.c", "-o", f"{d}/x"], check=True, stderr=sys.stderr)
        out = subprocess.run([f"{d}/x"], capture_output=True, text=True, check=True).stdout.split()
    assert [int(x) for x in out] == [ctypes.sizeof(kv.fakv_qcache)] + [getattr(kv.fakv_qcache, n).offset for n in fields]


@pytest.mark.parametrize("kw,code", [
    (dict(bits=5), 2), (dict(bits=0), 2), (dict(group=32), 2), (dict(group=0), 1), (dict(D=96, group=64), 2), (dict(D=136, group=136), 2),
    (dict(D=24, group=24), 2), (dict(page_size=4), 2), (dict(page_size=24), 2), (dict(page_size=2048), 2), (dict(dtype=7), 1),
    (dict(planes=0), 1), (dict(num_pages=0), 1), (dict(HKV=0), 1), (dict(max_slots=0), 1), (dict(max_pages=0), 1),
    (dict(K=0), 1), (dict(V=0), 1), (dict(table=0), 1), (dict(lens=0), 1), (dict(K=A + 8), 3), (dict(V=A + 4), 3), (dict(table=A + 2), 3),
    (dict(lens=A + 1), 3), (dict(status=A + 2), 3), (dict(head_stride=1024), 1), (dict(head_stride=1152 + 8), 3), (dict(head_stride=-1152), 1),
    (dict(page_stride=2304 + 4), 3), (dict(page_stride=0), 1), (dict(plane_stride=8), 3), (dict(plane_stride=0), 1),
    (dict(table_stride=7), 1), (dict(max_pages=1 << 27, table_stride=1 << 27), 1), (dict(page_stride=1 << 51), 1)])
def test_caches_that_are_refused(kv, kw, code):
    c = cache(kv, **kw)
    assert calls(kv, c, tokens(kv)) == (code,) * 3
    lib, C = kv._lib(), ctypes.byref(c)
    for f in (lib.fakv_qgrow, lib.fakv_qfork):
        assert f(C, A, A, 1, None) == code
    assert lib.fakv_qfree(C, A, None, 1, None) == code and lib.fakv_qcompact(C, None) == code


def test_block_sizes(kv):
    f = kv._lib().fakv_qblock_bytes
    assert f(16, 128, 4, 64) == 16 * 72 and f(8, 128, 8, 128) == 8 * 132 and f(1024, 16, 4, 16) == 1024 * 20
    assert f(32, 80, 4, 80) == 32 * (48 + 4) and f(32, 80, 8, 80) == 32 * 84
    for bad in ((12, 128, 4, 64), (16, 0, 4, 0), (16, 128, 3, 64), (16, 128, 4, 0), (16, 128, 4, 32), (16, 64, 4, 32), (16, -16, 4, -16)):
        assert f(*bad) == 0
    with pytest.raises(ValueError):
        kv.QuantCache.block_bytes(16, 128, 6)


def test_calls_that_are_refused(kv):
    lib = kv._lib()
    c = cache(kv)
    C = ctypes.byref(c)
    for kw in (dict(B=-1), dict(T=-1), dict(plane=3), dict(plane=-1), dict(B=16385), dict(T=1 << 30, H=4)):
        r = calls(kv, c, tokens(kv, **kw))
        assert r[0] == r[1] == 1, kw
        assert r[2] == 1 or kw.get("T") == 1 << 30 and r[2] == 1, kw
    for kw in (dict(H=3), dict(H=-2), dict(H=258), dict(q_token=-128), dict(k_head=-1)):
        assert calls(kv, c, tokens(kv, **kw))[:2] == (1, 1), kw
    for kw, code in ((dict(H=0), 1), (dict(scale=0.0), 1), (dict(scale=float("nan")), 1), (dict(scale=-1.0), 1), (dict(scale=3e38), 1),
                     (dict(causal=2), 1), (dict(window=-1), 1), (dict(out_dtype=2), 1), (dict(q_token=516), 3), (dict(q_head=4), 3)):
        assert lib.fakv_qattend(A, A, A, A, None, C, ctypes.byref(tokens(kv, **kw)), None) == code, kw
    P = ctypes.byref(tokens(kv))
    for i in range(3):
        for bad, code in ((0, 1), (A + 8, 3)):
            p = [A] * 3
            p[i] = bad
            assert lib.fakv_qattend(*p, A, None, C, P, None) == code
    for i in range(2):
        for bad, code in ((0, 1), (A + 8, 3)):
            p = [A] * 2
            p[i] = bad
            assert lib.fakv_qread(*p, A, None, None, C, P, None) == code
    assert lib.fakv_qread(A, A, 0, None, None, C, P, None) == 1 and lib.fakv_qread(A, A, A + 2, None, None, C, P, None) == 3
    assert lib.fakv_qread(A, A, A, A + 1, None, C, P, None) == 3 and lib.fakv_qread(A, A, A, None, A + 2, C, P, None) == 3
    assert lib.fakv_qread(A, A, A, None, None, C, ctypes.byref(tokens(kv, out_dtype=5)), None) == 1
    for i in range(5):
        p = [A] * 5
        p[i] = 0
        assert lib.fakv_qappend(*p, None, None, C, P, None) == 1
    assert lib.fakv_qappend(A, A + 1, A, A, A, None, None, C, P, None) == 3
    assert lib.fakv_qappend(A, A, A, A, A, None, None, C, ctypes.byref(tokens(kv, q_token=1024)), None) == 1  # in place, with gaps
    assert lib.fakv_qappend(A, A, A, A, A, None, ctypes.byref(kv.fakv_rope(A, 130, 0, 1.0)), C, P, None) == 1
    for f in (lib.fakv_qattend, lib.fakv_qread):
        assert f(A, A, A, A, None, None, P, None) == 1 and f(A, A, A, A, None, C, None, None) == 1
    assert lib.fakv_qappend(A, A, A, A, A, None, None, None, P, None) == 1
    # nothing to do
    assert calls(kv, c, tokens(kv, B=0)) == calls(kv, c, tokens(kv, T=0)) == (0, 0, 0)
    # the page calls' own
    for f in (lib.fakv_qgrow, lib.fakv_qfork):
        assert f(C, 0, A, 1, None) == f(C, A, 0, 1, None) == f(C, A, A, -1, None) == f(C, A, A, 16385, None) == 1
        assert f(C, A + 1, A, 1, None) == 3 and f(C, 0, 0, 0, None) == 0
    assert lib.fakv_qfree(C, 0, None, 1, None) == 1 and lib.fakv_qfree(C, A, A + 1, 1, None) == 3
    for kw, code in ((dict(refs=0), 1), (dict(head_stride=1152 + 16, page_stride=4096), 2), (dict(page_stride=1152), 1)):
        C2 = ctypes.byref(cache(kv, **kw))
        assert lib.fakv_qcompact(C2, None) == code and lib.fakv_qgrow(C2, A, A, 1, None) == code


def test_the_binding_refuses_before_it_calls(kv):
    if torch.cuda.is_available():
        pytest.skip("the checks on a CUDA device are with the GPU tests")
    z = torch.zeros(1, 4, 2, 16 * 72, dtype=torch.uint8)
    t, l, r = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    for a in ((z[..., :-1], z[..., :-1]), (z.float(), z.float()), (z, z[:, :3]), (z[0, 0], z[0, 0])):
        with pytest.raises(ValueError):
            kv.QuantCache(*a, t, l, r, 16, 128)
    with pytest.raises(TypeError):
        kv.QuantCache(z, z, t, l, r, 16, 128, dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        kv.QuantCache(z, z, t, l, r, 16, 128)
