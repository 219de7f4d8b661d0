"""Host-side checks of the q8kv boundary: no GPU, no kernel launches."""
import ctypes
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "q8kv.h")


@pytest.fixture(scope="session")
def q8():
    import __graft_entry__

    __graft_entry__._load_build_module().build_library()
    import q8_matrix_vector_gb300 as q8mv

    return q8mv


@pytest.fixture(scope="session")
def kv(q8):
    q8.Cache
    from q8_matrix_vector_gb300 import kv

    return kv


def declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(q8kv_[a-z_0-9]+)\s*\(", text)))


def test_every_declared_entry_point_is_exported_and_no_other(q8):
    out = subprocess.run(["nm", "-D", "--defined-only", q8.LIB], check=True, capture_output=True, text=True).stdout
    ours = sorted(s for s in (line.split()[-1] for line in out.splitlines() if line.strip()) if s.startswith("q8kv_"))
    assert ours == declared() and len(ours) == 11


def test_structures_match_the_header(kv, tmp_path):
    src = tmp_path / "sizes.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "q8kv.h"\nint main(void) { printf("%zu %zu %zu %zu %zu",'
                   "sizeof(q8kv_cache_t), sizeof(q8kv_attend_args_t), sizeof(q8kv_verify_args_t),"
                   "offsetof(q8kv_attend_args_t, scale), offsetof(q8kv_verify_args_t, type)); return 0; }\n")
    exe = tmp_path / "sizes"
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-I", cuda, str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert got == [ctypes.sizeof(kv.CacheDesc), ctypes.sizeof(kv.AttendArgs), ctypes.sizeof(kv.VerifyArgs),
                   kv.AttendArgs.scale.offset, kv.VerifyArgs.type.offset]


def desc(kv, **over):
    d = dict(k_codes=4096, k_scales=4096, v_codes=4096, v_scales=4096, pages=4, page_size=16, heads=2, head_dim=64,
             reserved=0, stride_page=32, stride_head=16, stride_token=1)
    d.update(over)
    return kv.CacheDesc(**d)


BAD_CACHES = [dict(k_codes=None), dict(v_scales=None), dict(k_codes=4104), dict(k_scales=4100), dict(pages=-1),
              dict(page_size=0), dict(page_size=65537), dict(heads=0), dict(head_dim=0), dict(head_dim=40),
              dict(head_dim=272), dict(reserved=1), dict(stride_page=0), dict(stride_head=-1), dict(stride_token=0),
              dict(pages=2 ** 31), dict(pages=2 ** 30, page_size=65536), dict(stride_page=2 ** 51)]


@pytest.mark.parametrize("over", BAD_CACHES)
def test_calls_refuse_a_bad_cache(q8, kv, over):
    lib, d = q8.library(), desc(kv, **over)
    assert lib.q8kv_cache_write(d, 1, 4096, 4096, 0, 128, 64, 128, 64, 4096, None) == q8.Q8MV_ERR_INVALID_ARG
    assert lib.q8kv_cache_read(d, 1, 4096, 4096, 4096, 0, None) == q8.Q8MV_ERR_INVALID_ARG
    assert lib.q8kv_cache_move(d, 1, 1, 4096, 4096, None) == q8.Q8MV_ERR_INVALID_ARG


def test_cache_calls_refuse_bad_arguments(q8, kv):
    lib, d, bad = q8.library(), desc(kv), q8.Q8MV_ERR_INVALID_ARG
    good = dict(n=1, k=4096, v=4096, type=0, kr=128, kh=64, vr=128, vh=64, slots=4096)
    for over in (dict(n=-1), dict(n=2 ** 31), dict(k=None), dict(v=None), dict(slots=None), dict(type=3), dict(type=-1),
                 dict(kr=-1), dict(vh=-64), dict(kh=2 ** 40), dict(k=4098), dict(slots=4100)):
        a = {**good, **over}
        assert lib.q8kv_cache_write(d, a["n"], a["k"], a["v"], a["type"], a["kr"], a["kh"], a["vr"], a["vh"], a["slots"],
                                    None) == bad, over
    for n, slots, k, v, t in ((-1, 4096, 4096, 4096, 0), (1, None, 4096, 4096, 0), (1, 4096, None, 4096, 0),
                              (1, 4096, 4096, 4104, 0), (1, 4097, 4096, 4096, 0), (1, 4096, 4096, 4096, 9)):
        assert lib.q8kv_cache_read(d, n, slots, k, v, t, None) == bad
    for batch, path, src, dst in ((-1, 1, 4096, 4096), (65536, 1, 4096, 4096), (1, -1, 4096, 4096), (1, 1, None, 4096),
                                  (1, 1, 4096, 4100)):
        assert lib.q8kv_cache_move(d, batch, path, src, dst, None) == bad
    # nothing to do
    assert lib.q8kv_cache_write(d, 0, None, None, 0, 0, 0, 0, 0, None, None) == q8.Q8MV_OK
    assert lib.q8kv_cache_read(d, 0, None, None, None, 0, None) == q8.Q8MV_OK
    assert lib.q8kv_cache_move(d, 0, 5, None, None, None) == q8.Q8MV_OK
    assert lib.q8kv_cache_move(d, 5, 0, None, None, None) == q8.Q8MV_OK


def test_plans_refuse_bad_sizes_before_touching_a_device(q8, kv):
    lib, bad = q8.library(), q8.Q8MV_ERR_INVALID_ARG
    for hq, hk, dim, b, r in ((0, 1, 64, 1, 1), (3, 2, 64, 1, 1), (2, 4, 64, 1, 1), (4, 2, 24, 1, 1), (4, 2, 512, 1, 1),
                              (4, 2, 64, 0, 1), (4, 2, 64, 1, 0), (4, 2, 64, 65537, 1), (4, 2, 64, 1, 2 ** 20 + 1),
                              (65534, 65534, 64, 65536, 2 ** 20)):
        h = ctypes.c_void_p(7)
        assert lib.q8kv_attend_plan(ctypes.byref(h), hq, hk, dim, b, r, -1) == bad
        assert h.value is None
    assert lib.q8kv_attend_plan(None, 4, 2, 64, 1, 1, -1) == bad
    for b, r, v in ((0, 1, 10), (1, 0, 10), (1, 1, 0), (65536, 1, 10), (1, 2 ** 20 + 1, 10), (1, 1, 2 ** 22 + 1)):
        h = ctypes.c_void_p(7)
        assert lib.q8kv_verify_plan(ctypes.byref(h), b, r, v, -1) == bad
        assert h.value is None
    assert lib.q8kv_verify_plan(None, 1, 1, 10, -1) == bad
    args = kv.AttendArgs()
    assert lib.q8kv_attend(None, desc(kv), ctypes.byref(args), None) == bad
    assert lib.q8kv_verify(None, ctypes.byref(kv.VerifyArgs()), None) == bad
    assert lib.q8kv_attend_destroy(None) == q8.Q8MV_OK and lib.q8kv_verify_destroy(None) == q8.Q8MV_OK


def test_plans_without_a_gpu_say_so(q8, kv):
    import torch

    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    with pytest.raises(q8.Q8mvError):
        q8.TreeAttention(4, 2, 64, 1, 1)
    with pytest.raises(q8.Q8mvError):
        q8.TreeVerify(1, 1, 100)
    with pytest.raises(ValueError):
        q8.Cache.of(*(torch.zeros(1, 1, 1, n, dtype=t) for n, t in
                      ((32, torch.int8), (1, torch.float32), (32, torch.int8), (1, torch.float32))))
