"""Host-only checks of include/fakv.h: exports, struct layouts, refusals (no call here reaches a kernel) and the
rotary frequencies."""
import ctypes
import math
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A, MIS = 0x10000, 0x10008  # never dereferenced


@pytest.fixture(scope="module")
def kv():
    import __graft_entry__
    __graft_entry__.build_library()
    from attention_fa_fwd_02_gb300 import kv as m
    return m


def test_every_declared_symbol_is_exported_and_no_other(kv):
    from attention_fa_fwd_02_gb300 import fa
    text = open(os.path.join(ROOT, "include", "fakv.h")).read()
    declared = set(re.findall(r"FA_API\s+[\w\s\*]*?\b(fakv_\w+)\s*\(", text))
    assert declared == set(kv.EXPORTS)
    out = os.popen(f"nm -D --defined-only {fa.LIB_PATH}").read()
    assert set(re.findall(r"\bT (\w+)", out)) - {"_init", "_fini"} == declared | set(fa.EXPORTS)


@pytest.mark.parametrize("name", ["fakv_cache", "fakv_scaling", "fakv_rope", "fakv_rope_params", "fakv_tokens"])
def test_struct_layouts_match_the_header(kv, name, tmp_path):
    cc = shutil.which("gcc")
    if cc is None:
        pytest.skip("needs gcc")
    t = getattr(kv, name)
    names = [n for n, _ in t._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "fakv.h"\nint main(void) {\n'
                   + f'  printf("%zu", sizeof({name}));\n'
                   + "".join(f'  printf(" %zu", offsetof({name}, {n}));\n' for n in names) + "  return 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()]
    assert got == [ctypes.sizeof(t)] + [getattr(t, n).offset for n in names]


def test_packed_parameters_are_the_structs(kv):
    for pack, t, values in (
            (kv._pack_tokens, kv.fakv_tokens, (1, 2, 3, 4, 5, 6, 7, 8, 9, 1 << 40, 0.5, 1, 12, 1)),
            (kv._pack_rope, kv.fakv_rope_params, (1, 2, 3, 4, 1, True, False, 8, 9, 10, 11, 12, 13, 14, 1 << 40))):
        b = pack(*values)
        assert len(b) == ctypes.sizeof(t)
        x = t.from_buffer_copy(b)
        assert [getattr(x, n) for n, _ in t._fields_] == [v for v in values]


def cache(kv, **kw):
    d = dict(K=A, V=A, table=A, lens=A, refs=A, status=0, plane_stride=0, page_stride=16 * 2 * 64, token_stride=128,
             head_stride=64, table_stride=10, planes=1, num_pages=100, page_size=16, HKV=2, D=64, max_slots=4,
             max_pages=10, dtype=1)
    d.update(kw)
    return kv.fakv_cache(**d)


def tokens(kv, **kw):
    d = dict(B=2, T=3, H=4, plane=0, q_token=256, q_head=64, k_token=128, k_head=64, v_token=128, v_head=64, scale=0.1,
             causal=1, window=0, out_dtype=1)
    d.update(kw)
    return kv.fakv_tokens(**d)


def calls(kv, c, t):
    lib, C, P = kv._lib(), ctypes.byref(c), ctypes.byref(t)
    return (lib.fakv_attend(A, A, A, A, None, C, P, None), lib.fakv_append(A, A, A, A, A, None, None, C, P, None))


@pytest.mark.parametrize("kw,code", [
    (dict(D=24), 2), (dict(D=144), 2), (dict(D=0), 1), (dict(page_size=4), 2), (dict(page_size=24), 2),
    (dict(page_size=2048), 2), (dict(page_size=0), 1), (dict(HKV=0), 1), (dict(num_pages=0), 1), (dict(planes=0), 1),
    (dict(max_slots=0), 1), (dict(max_pages=0), 1), (dict(dtype=2), 1), (dict(K=0), 1), (dict(V=0), 1),
    (dict(table=0), 1), (dict(lens=0), 1), (dict(K=MIS), 3), (dict(V=MIS), 3), (dict(lens=A + 2), 3),
    (dict(token_stride=0), 1), (dict(page_stride=-2048), 1), (dict(head_stride=60), 3), (dict(token_stride=129), 3),
    (dict(table_stride=9), 1), (dict(max_pages=1 << 27, table_stride=1 << 27), 1), (dict(num_pages=1 << 29), 1),
    (dict(planes=2, plane_stride=0), 1), (dict(planes=2, plane_stride=1 << 52), 1), (dict(page_stride=1 << 48), 1),
])
def test_bad_caches_are_refused(kv, kw, code):
    c = cache(kv, **kw)
    assert calls(kv, c, tokens(kv)) == (code, code)
    lib, C = kv._lib(), ctypes.byref(c)
    assert lib.fakv_grow(C, A, A, 1, None) == code
    assert lib.fakv_fork(C, A, A, 1, None) == code
    assert lib.fakv_free(C, A, None, 1, None) == code
    assert lib.fakv_compact(C, None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), 1), (dict(B=16385), 1), (dict(T=-1), 1), (dict(H=3), 1), (dict(H=2 * 129), 1), (dict(plane=1), 1),
    (dict(plane=-1), 1), (dict(q_token=-8), 1), (dict(q_token=1 << 50), 1), (dict(T=1 << 29), 1)])
def test_bad_tokens_are_refused(kv, kw, code):
    assert calls(kv, cache(kv), tokens(kv, **kw)) == (code, code)


def test_refusals_of_attend_and_append_alone(kv):
    lib, c = kv._lib(), cache(kv)
    C = ctypes.byref(c)
    for kw, code in ((dict(scale=0.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(scale=3e38), 1),
                     (dict(causal=2), 1), (dict(window=-1), 1), (dict(out_dtype=5), 1), (dict(H=0), 1),
                     (dict(q_head=60), 3), (dict(q_token=257), 3)):
        assert lib.fakv_attend(A, A, A, A, None, C, ctypes.byref(tokens(kv, **kw)), None) == code
    t = tokens(kv)
    P = ctypes.byref(t)
    for i in range(4):
        p = [A] * 4
        p[i] = 0
        assert lib.fakv_attend(*p, None, C, P, None) == 1
        if i < 3:
            p[i] = MIS
            assert lib.fakv_attend(*p, None, C, P, None) == 3
    assert lib.fakv_attend(A, A, A, A, A + 2, C, P, None) == 3
    for i in range(5):
        p = [A, A, A, A + 64, A]
        p[i] = 0
        assert lib.fakv_append(*p, None, None, C, P, None) == 1
    assert lib.fakv_append(A, A + 1, A, A, A, None, None, C, P, None) == 3
    # q rotated in place must be contiguous
    assert lib.fakv_append(A, A, A, A, A, None, None, C, ctypes.byref(tokens(kv, q_token=512)), None) == 1
    bad = kv.fakv_rope(A, 66, 0, 1.0)
    assert lib.fakv_append(A, A, A, A, A, None, ctypes.byref(bad), C, P, None) == 1
    assert lib.fakv_attend(A, A, A, A, None, None, P, None) == 1
    assert lib.fakv_attend(A, A, A, A, None, C, None, None) == 1
    # nothing to do: no pointer is touched
    assert lib.fakv_attend(0, 0, 0, 0, None, C, ctypes.byref(tokens(kv, T=0)), None) == 0
    assert lib.fakv_append(0, 0, 0, 0, 0, None, None, C, ctypes.byref(tokens(kv, B=0)), None) == 0


def test_refusals_of_the_page_calls(kv):
    lib = kv._lib()
    C = ctypes.byref(cache(kv))
    for f in (lib.fakv_grow, lib.fakv_fork):
        assert f(C, A, A, -1, None) == 1 and f(C, A, A, 16385, None) == 1
        assert f(C, 0, A, 1, None) == 1 and f(C, A, 0, 1, None) == 1
        assert f(C, A + 2, A, 1, None) == 3
        assert f(C, 0, 0, 0, None) == 0
    assert lib.fakv_free(C, 0, None, 1, None) == 1 and lib.fakv_free(C, A, A + 1, 1, None) == 3
    assert lib.fakv_free(C, 0, None, 0, None) == 0
    wide = cache(kv, max_pages=1 << 20, table_stride=1 << 20)
    assert lib.fakv_fork(ctypes.byref(wide), A, A, 4096, None) == 1  # too many rows to hold at once
    for kw, code in ((dict(refs=0), 1), (dict(token_stride=256), 2), (dict(page_stride=1024), 1)):
        assert lib.fakv_compact(ctypes.byref(cache(kv, **kw)), None) == code
        assert lib.fakv_grow(ctypes.byref(cache(kv, **kw)), A, A, 1, None) == code


def test_refusals_of_rope_apply(kv):
    lib = kv._lib()

    def call(ptrs=(A, A, A, A, A), rope=None, **kw):
        d = dict(T=3, H=4, HKV=2, D=64, dtype=1, positions_64=1, inverse=0, q_token=256, q_head=64, k_token=128,
                 k_head=64, qo_token=256, qo_head=64, ko_token=128, ko_head=64)
        d.update(kw)
        r = rope or kv.fakv_rope(A, 64, 0, 1.0)
        return lib.fakv_rope_apply(*ptrs, ctypes.byref(r), ctypes.byref(kv.fakv_rope_params(**d)), None)

    for kw, code in ((dict(T=-1), 1), (dict(H=0), 1), (dict(HKV=-1), 1), (dict(D=40), 2), (dict(D=160), 2),
                     (dict(dtype=3), 1), (dict(positions_64=2), 1), (dict(inverse=2), 1), (dict(q_token=-1), 1),
                     (dict(H=1 << 17), 1), (dict(qo_token=512), 1), (dict(ko_head=128), 1)):
        assert call(**kw) == code, kw
    for i in range(5):
        p = [A] * 5
        p[i] = 0
        assert call(p) == 1
    assert call((A, A, A, A, A + 4)) == 3 and call((A + 1, A, A, A, A)) == 3
    for r in (kv.fakv_rope(0, 64, 0, 1.0), kv.fakv_rope(A, 0, 0, 1.0), kv.fakv_rope(A, 63, 0, 1.0),
              kv.fakv_rope(A, 66, 0, 1.0), kv.fakv_rope(A, 64, 2, 1.0), kv.fakv_rope(A, 64, 0, float("nan"))):
        assert call(rope=r) == 1
    assert call((0, 0, 0, 0, 0), T=0) == 0


@pytest.mark.parametrize("rot,base,scaling", [
    (128, 10000.0, None), (2, 10000.0, None), (64, 500000.0, dict(kind="linear", factor=4.0)),
    (96, 10000.0, dict(kind="ntk", factor=8.0)),
    (128, 500000.0, dict(kind="bands", factor=8.0, low=1.0, high=4.0, original=8192)),
    (64, 10000.0, dict(kind="yarn", factor=16.0, beta_fast=32.0, beta_slow=1.0, original=4096)),
    (64, 10000.0, dict(kind="linear", factor=0.01))])  # a frequency above a turn a token
def test_frequencies_are_fractions_of_a_turn(kv, rot, base, scaling):
    import _kv_ref as ref
    r = kv.Rope(128, rot, base, scaling=scaling, device="cpu")
    want, m = ref.freqs(rot, base, scaling)
    assert abs(r.mscale - m) < 1e-6 and r.freqs.shape == (rot // 2,)
    for got, f in zip(r.freqs.tolist(), want):
        turns = (got % (1 << 64)) / 2.0 ** 64
        # pow, the scaling and the division by 2 pi: a few 2^-53 of f
        d = abs(turns - f / (2 * math.pi) % 1.0)
        assert min(d, 1 - d) <= 16 * 2.0 ** -53 * max(f, 2.0 ** -11)


def test_rope_refuses_bad_scalings(kv):
    from attention_fa_fwd_02_gb300 import fa
    for kw in (dict(kind="linear", factor=0.0), dict(kind="linear", factor=float("nan")),
               dict(kind="bands", factor=8.0, low=4.0, high=4.0, original=8192),
               dict(kind="bands", factor=8.0, low=1.0, high=4.0), dict(kind="yarn", factor=4.0, original=-1.0),
               dict(kind="yarn", factor=4.0, original=4096, beta_fast=1.0, beta_slow=1.0)):
        with pytest.raises(fa.FAError):
            kv.Rope(128, scaling=kw, device="cpu")
    with pytest.raises(ValueError):
        kv.Rope(128, scaling=dict(kind="cubic"), device="cpu")
    with pytest.raises(ValueError):
        kv.Rope(128, scaling=dict(kind="linear", factor=2.0, power=3.0), device="cpu")
    with pytest.raises(ValueError):
        kv.Rope(64, 128, device="cpu")
    with pytest.raises(fa.FAError):
        kv.Rope(64, 63, device="cpu")
    with pytest.raises(fa.FAError):
        kv.Rope(64, 2, scaling=dict(kind="ntk", factor=2.0), device="cpu")
    with pytest.raises(fa.FAError):
        kv.Rope(64, base=1.0, device="cpu")


def test_the_binding_refuses_what_it_can_see(kv):
    import torch
    z = torch.zeros
    with pytest.raises(ValueError):  # not on a GPU
        kv.PagedCache(z(1, 2, 16, 1, 64), z(1, 2, 16, 1, 64), z(1, 2).int(), z(1).int(), z(2).int())
    with pytest.raises(ValueError):
        kv.PagedCache(z(1, 2, 16, 1, 64), z(1, 2, 16, 1, 32), z(1, 2).int(), z(1).int(), z(2).int())
    r = kv.Rope(64, device="cpu")
    with pytest.raises(ValueError):
        r.apply(z(2, 1, 64), None, z(2).long())
    with pytest.raises(ValueError):
        r.apply(z(2, 1, 32), None, z(2).long())


def test_what_no_launch_could_take_is_refused(kv):
    c, t = cache(kv, HKV=1000, token_stride=64000, page_stride=16 * 64000), tokens(kv, H=66000, T=1, B=1)
    assert calls(kv, c, t) == (1, 1)  # more heads than a grid has rows of blocks
    with pytest.raises(ValueError):   # a scaling without its kind
        kv.Rope(64, scaling=dict(factor=2.0), device="cpu")
