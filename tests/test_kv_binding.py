"""The q8kv binding on the host: reached by any import, and what its checks refuse."""
import os
import subprocess
import sys

import pytest

from test_kv_host import kv, q8  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("how", ["from q8_matrix_vector_gb300 import kv", "import q8_matrix_vector_gb300.kv as kv",
                                 "from q8_matrix_vector_gb300 import Cache; from q8_matrix_vector_gb300 import kv"])
def test_the_entry_points_are_declared_however_the_module_is_imported(q8, how):  # noqa: F811
    """Without declared arguments ctypes passes the lower 32 bits of a pointer."""
    code = how + "\nlib = kv._library()\nassert all(getattr(lib, n).argtypes for n in %r)" % (
        ["q8kv_cache_write", "q8kv_cache_read", "q8kv_cache_move", "q8kv_attend_plan", "q8kv_attend", "q8kv_attend_check",
         "q8kv_attend_set_wait", "q8kv_attend_destroy", "q8kv_verify_plan", "q8kv_verify", "q8kv_verify_destroy"],)
    subprocess.run([sys.executable, "-c", code], check=True, cwd=ROOT)


@pytest.mark.parametrize("over", [dict(heads=65535, stride_head=2 ** 48), dict(heads=2, stride_head=2 ** 52),
                                  dict(page_size=65536, stride_token=2 ** 48), dict(page_size=16, stride_token=2 ** 49),
                                  dict(stride_page=2 ** 62), dict(stride_head=2 ** 62), dict(stride_token=2 ** 62),
                                  dict(pages=1, stride_page=2 ** 53)])
def test_a_cache_whose_rows_pass_63_bits_is_refused(q8, kv, over):  # noqa: F811
    """Products of strides and counts, as the checks behind this one form them, stay numbers."""
    from test_kv_host import desc

    lib, d = q8.library(), desc(kv, **over)
    assert lib.q8kv_cache_write(d, 0, None, None, 0, 0, 0, 0, 0, None, None) == q8.Q8MV_ERR_INVALID_ARG
    assert lib.q8kv_cache_read(d, 0, None, None, None, 0, None) == q8.Q8MV_ERR_INVALID_ARG
    assert lib.q8kv_cache_move(d, 0, 0, None, None, None) == q8.Q8MV_ERR_INVALID_ARG
