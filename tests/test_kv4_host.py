"""Host-side checks of the q4kv, kvrope and kvpage boundaries: no GPU, no kernel launches."""
import ctypes
import os
import re
import subprocess
import sys

import pytest

from test_kv_host import q8  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADERS = {"q4kv.h": ("q4kv_", 8), "kvrope.h": ("kvrope_", 5), "kvpage.h": ("kvpage_", 8)}


@pytest.fixture(scope="session")
def mods(q8):  # noqa: F811
    q8.Cache4, q8.Rotary, q8.Pages
    from q8_matrix_vector_gb300 import kv, kv4, pages, rotary

    return kv, kv4, rotary, pages


@pytest.mark.parametrize("header", sorted(HEADERS))
def test_every_declared_entry_point_is_exported_and_no_other(q8, header):  # noqa: F811
    prefix, count = HEADERS[header]
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    declared = sorted(set(re.findall(r"\b(%s[a-z_0-9]+)\s*\(" % prefix, text)))
    out = subprocess.run(["nm", "-D", "--defined-only", q8.LIB], check=True, capture_output=True, text=True).stdout
    ours = sorted(s for s in (line.split()[-1] for line in out.splitlines() if line.strip()) if s.startswith(prefix))
    assert ours == declared and len(ours) == count


def test_structures_match_the_headers(mods, tmp_path):
    kv, _, rotary, pages = mods
    src = tmp_path / "sizes.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "kvrope.h"\n#include "kvpage.h"\nint main(void) { '
                   'printf("%zu %zu %zu %zu %zu %zu %zu", sizeof(q4kv_cache_t), offsetof(q4kv_cache_t, stride_page),'
                   "sizeof(kvrope_write_args_t), offsetof(kvrope_write_args_t, positions), offsetof(kvrope_write_args_t, type),"
                   "sizeof(kvpage_state_t), offsetof(kvpage_state_t, held)); return 0; }\n")
    exe = tmp_path / "sizes"
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    subprocess.run(["gcc", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-I", cuda, str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert got == [ctypes.sizeof(kv.CacheDesc), kv.CacheDesc.stride_page.offset, ctypes.sizeof(rotary.WriteArgs),
                   rotary.WriteArgs.positions.offset, rotary.WriteArgs.type.offset, ctypes.sizeof(pages.State),
                   pages.State.held.offset]


@pytest.mark.parametrize("how", ["from q8_matrix_vector_gb300 import kv4", "from q8_matrix_vector_gb300 import Cache4",
                                 "import q8_matrix_vector_gb300 as q; q.TreeAttention4"])
def test_the_entry_points_are_declared_however_the_module_is_imported(q8, how):  # noqa: F811
    code = how + "\nfrom q8_matrix_vector_gb300 import kv\nlib = kv._library()\nassert all(getattr(lib, n).argtypes for n in %r)" % (
        ["q4kv_cache_write", "q4kv_cache_read", "q4kv_cache_move", "q4kv_attend_plan", "q4kv_attend", "q4kv_attend_check",
         "q4kv_attend_set_wait", "q4kv_attend_destroy", "kvpage_copy_q4", "kvpage_copy_q8"],)
    subprocess.run([sys.executable, "-c", code], check=True, cwd=ROOT)
    for name, names in (("Rotary", ["kvrope_plan", "kvrope_apply", "kvrope_write_q8", "kvrope_write_q4", "kvrope_destroy"]),
                        ("Pages", ["kvpage_plan", "kvpage_extend", "kvpage_fork", "kvpage_free", "kvpage_compact"])):
        code = "import q8_matrix_vector_gb300 as q; q.%s\nassert all(getattr(q._lib, n).argtypes for n in %r)" % (name, names)
        subprocess.run([sys.executable, "-c", code], check=True, cwd=ROOT)


def desc(mods, **over):
    d = dict(k_codes=4096, k_scales=4096, v_codes=4096, v_scales=4096, pages=4, page_size=16, heads=2, head_dim=64,
             reserved=0, stride_page=32, stride_head=16, stride_token=1)
    d.update(over)
    return mods[0].CacheDesc(**d)


BAD = [dict(k_codes=None), dict(v_scales=None), dict(k_codes=4104), dict(k_scales=4100), dict(pages=-1), dict(page_size=0),
       dict(page_size=65537), dict(heads=0), dict(head_dim=0), dict(head_dim=40), dict(head_dim=272), dict(reserved=1),
       dict(stride_page=0), dict(stride_head=-1), dict(stride_token=0), dict(pages=2 ** 31),
       dict(pages=2 ** 30, page_size=65536), dict(stride_page=2 ** 51), dict(stride_head=2 ** 62)]


@pytest.mark.parametrize("over", BAD)
def test_calls_refuse_a_bad_cache(q8, mods, over):  # noqa: F811
    lib, d = q8.library(), desc(mods, **over)
    no = q8.Q8MV_ERR_INVALID_ARG
    assert lib.q4kv_cache_write(d, 1, 4096, 4096, 0, 128, 64, 128, 64, 4096, None) == no
    assert lib.q4kv_cache_read(d, 1, 4096, 4096, 4096, 0, None) == no
    assert lib.q4kv_cache_move(d, 1, 1, 4096, 4096, None) == no
    assert lib.kvpage_copy_q4(d, 1, 4096, 4096, None, None) == no
    assert lib.kvpage_copy_q8(d, 1, 4096, 4096, None, None) == no
    # a cache of nothing may have null pointers, whatever the calls are about to do
    assert lib.q4kv_cache_write(desc(mods, pages=0, k_codes=None), 1, 4096, 4096, 0, 1, 1, 1, 1, 4096, None) == q8.Q8MV_OK


@pytest.mark.parametrize("args", [(-1, 4096, 4096, 0, 1, 1, 1, 1, 4096), (2 ** 31, 4096, 4096, 0, 1, 1, 1, 1, 4096),
                                  (1, None, 4096, 0, 1, 1, 1, 1, 4096), (1, 4096, None, 0, 1, 1, 1, 1, 4096),
                                  (1, 4098, 4096, 0, 1, 1, 1, 1, 4096), (1, 4097, 4096, 1, 1, 1, 1, 1, 4096),
                                  (1, 4096, 4096, 3, 1, 1, 1, 1, 4096), (1, 4096, 4096, -1, 1, 1, 1, 1, 4096),
                                  (1, 4096, 4096, 0, -1, 1, 1, 1, 4096), (1, 4096, 4096, 0, 1, 2 ** 40, 1, 1, 4096),
                                  (1, 4096, 4096, 0, 1, 1, 1, 1, None), (1, 4096, 4096, 0, 1, 1, 1, 1, 4100)])
def test_write_refuses(q8, mods, args):  # noqa: F811
    assert q8.library().q4kv_cache_write(desc(mods), *args, None) == q8.Q8MV_ERR_INVALID_ARG


def test_read_move_and_copies_refuse(q8, mods):  # noqa: F811
    lib, d, no = q8.library(), desc(mods), q8.Q8MV_ERR_INVALID_ARG
    for args in ((-1, 4096, 4096, 4096, 0), (1, None, 4096, 4096, 0), (1, 4096, 4104, 4096, 0), (1, 4096, 4096, None, 0),
                 (1, 4096, 4096, 4096, 5), (1, 4100, 4096, 4096, 0)):
        assert lib.q4kv_cache_read(d, *args, None) == no
    for args in ((-1, 1, 4096, 4096), (65536, 1, 4096, 4096), (1, -1, 4096, 4096), (1, 1, None, 4096), (1, 1, 4096, 4100)):
        assert lib.q4kv_cache_move(d, *args, None) == no
    for args in ((-1, 4096, 4096, None), (2 ** 31, 4096, 4096, None), (1, None, 4096, None), (1, 4096, None, None),
                 (1, 4098, 4096, None), (1, 4096, 4096, 4097)):
        assert lib.kvpage_copy_q4(d, *args, None) == no and lib.kvpage_copy_q8(d, *args, None) == no
    # a page of more pieces than 31 bits number
    big = desc(mods, heads=65535, page_size=65536, head_dim=256, pages=1)
    assert lib.kvpage_copy_q4(big, 1, 4096, 4096, None, None) == no
    # nothing to do
    assert lib.q4kv_cache_read(d, 0, None, None, None, 0, None) == q8.Q8MV_OK
    assert lib.q4kv_cache_move(d, 0, 5, None, None, None) == q8.Q8MV_OK
    assert lib.kvpage_copy_q4(d, 0, None, None, None, None) == q8.Q8MV_OK


def test_plans_refuse(q8, mods):  # noqa: F811
    lib, no, h = q8.library(), q8.Q8MV_ERR_INVALID_ARG, ctypes.c_void_p()
    for args in ((0, 1, 64, 1, 1), (4, 0, 64, 1, 1), (4, 3, 64, 1, 1), (2, 4, 64, 1, 1), (4, 2, 72, 1, 1), (4, 2, 272, 1, 1),
                 (4, 2, 64, 0, 1), (4, 2, 64, 65537, 1), (4, 2, 64, 1, 0), (4, 2, 64, 1, 2 ** 20 + 1),
                 (65535, 65535, 64, 65536, 1)):
        assert lib.q4kv_attend_plan(ctypes.byref(h), *args, -1) == no and not h.value
    turns = (ctypes.c_uint64 * 32)()
    for args in ((64, 3, 0, turns, 1.0), (64, 66, 0, turns, 1.0), (64, 0, 0, turns, 1.0), (1, 2, 0, turns, 1.0),
                 (70000, 64, 0, turns, 1.0), (1024, 514, 0, turns, 1.0), (64, 64, 2, turns, 1.0), (64, 64, 0, None, 1.0),
                 (64, 64, 0, turns, float("inf")), (64, 64, 0, turns, float("nan"))):
        assert lib.kvrope_plan(ctypes.byref(h), *args, -1) == no and not h.value
    for args in ((0, 16, 1, 1), (2 ** 28 + 1, 16, 1, 1), (1, 0, 1, 1), (1, 65537, 1, 1), (1, 16, 0, 1), (1, 16, 65536, 1),
                 (1, 16, 1, 0), (1, 16, 1, 2 ** 24 + 1), (1, 16, 2 ** 15, 2 ** 14)):
        assert lib.kvpage_plan(ctypes.byref(h), *args, -1) == no and not h.value
    for f in (lib.q4kv_attend_plan, ):
        assert f(None, 4, 2, 64, 1, 1, -1) == no
    assert lib.kvrope_plan(None, 64, 64, 0, turns, 1.0, -1) == no and lib.kvpage_plan(None, 1, 1, 1, 1, -1) == no


def test_calls_refuse_no_plan(q8, mods):  # noqa: F811
    lib, no = q8.library(), q8.Q8MV_ERR_INVALID_ARG
    d, word = desc(mods), ctypes.c_int32()
    assert lib.q4kv_attend(None, d, ctypes.create_string_buffer(256), None) == no
    assert lib.q4kv_attend_check(None, ctypes.byref(word)) == no and lib.q4kv_attend_set_wait(None, 0) == no
    assert lib.kvrope_apply(None, 1, 1, 0, 4096, 64, 64, 4096, 4096, 64, 64, 0, None) == no
    assert lib.kvrope_write_q8(None, d, ctypes.create_string_buffer(256), None) == no
    assert lib.kvrope_write_q4(None, d, ctypes.create_string_buffer(256), None) == no
    state = mods[3].State(4096, 4096, 4096)
    assert lib.kvpage_extend(None, state, 4096, 4096, 1, 4096, 4096, 4096, 4096, None) == no
    assert lib.kvpage_fork(None, state, 4096, None) == no and lib.kvpage_free(None, state, 4096, None) == no
    assert lib.kvpage_compact(None, state, 4096, 4096, 4096, None) == no
    # no plan to release
    assert lib.q4kv_attend_destroy(None) == q8.Q8MV_OK and lib.kvrope_destroy(None) == q8.Q8MV_OK
    assert lib.kvpage_destroy(None) == q8.Q8MV_OK


def test_frequencies():
    """The rules of scaling at their ends: the fastest pairs stay, the slowest are divided by the factor."""
    from q8_matrix_vector_gb300.rotary import frequencies

    plain, one = frequencies(128)
    assert one == 1.0 and plain[0] == 1.0 and abs(plain[-1] * 10000.0 ** (126 / 128) - 1) < 1e-12
    linear, one = frequencies(128, scaling=dict(kind="linear", factor=8.0))
    assert one == 1.0 and all(abs(8 * a / b - 1) < 1e-12 for a, b in zip(linear, plain))
    ntk, _ = frequencies(128, scaling=dict(kind="ntk", factor=8.0))
    assert ntk[0] == 1.0 and abs(8 * ntk[-1] / plain[-1] - 1) < 1e-12
    yarn, attention = frequencies(128, scaling=dict(kind="yarn", factor=8.0, original=4096))
    assert yarn[0] == plain[0] and abs(8 * yarn[-1] / plain[-1] - 1) < 1e-12 and abs(attention - 1.2079441541679836) < 1e-12
    assert all(a <= b for a, b in zip(yarn, plain)) and yarn == sorted(yarn, reverse=True)
    bands, one = frequencies(128, scaling=dict(kind="bands", factor=8.0, original=8192, low=1.0, high=4.0))
    assert one == 1.0
    for b, f in zip(bands, plain):
        turns = 8192 * f / (2 * 3.141592653589793)
        assert abs(b / f - (1 if turns >= 4 else 0.125 if turns <= 1 else (turns - 1) / 3 + 0.125 * (4 - turns) / 3)) < 1e-12


def test_the_plain_pool_keeps_its_counts():
    """The reference's own invariant: refs are what the tables hold."""
    import numpy as np

    import kv4_ref as ref

    rng = np.random.default_rng(0)
    pool = ref.Pool(50, 4, 5, 12)
    lengths = np.zeros(5, int)
    for _ in range(50):
        tokens = rng.integers(0, 9, 5)
        _, src, dst, ok = pool.extend(lengths, tokens, 9)
        lengths = np.where(ok == 1, lengths + tokens, lengths)
        parents = rng.integers(-1, 5, 5)
        pool.fork(parents)
        lengths = np.where(parents >= 0, lengths[parents], 0)
        pool.free(lengths)
        if rng.random() < 0.3:
            pool.compact()
        counts = np.zeros(50, int)
        for b in range(5):
            for c in range(pool.held[b]):
                counts[pool.table[b, c]] += 1
            assert (pool.table[b, pool.held[b]:] == -1).all()
        assert np.array_equal(counts, pool.refs)


def test_packing_is_its_own_inverse():
    import numpy as np

    import kv4_ref as ref

    rng = np.random.default_rng(1)
    for dim in (64, 80, 128, 192, 256):
        nb = ref.blocks4(dim)
        codes = rng.integers(0, 16, (3, 32 * nb)).astype(np.uint8)
        for unit in (2, 4):
            row = ref.pack(codes, unit)
            assert row.shape == (3, 16 * nb)
            for e in rng.integers(0, 32 * nb, 40):
                b, i = e // 32, e % 32
                byte = row[:, unit * (i // 2 // unit * nb + b) + i // 2 % unit]
                assert np.array_equal(byte >> (4 * (i & 1)) & 15, codes[:, e])
