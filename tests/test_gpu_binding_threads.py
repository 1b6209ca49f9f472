"""The native part of the binding from several Python threads."""
import ctypes
import shutil
import subprocess
import threading
import time

import pytest
import torch

from test_gpu_window import P  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


@pytest.fixture
def slow_library(P, tmp_path):  # noqa: F811
    """The binding over a library whose calls take 0.3 s on the host, as one does whose
    launch waits for room in the stream's queue."""
    if not shutil.which("g++"):
        pytest.skip("g++ not available")
    src, so = tmp_path / "slow.cpp", tmp_path / "slow.so"
    src.write_text('#include <unistd.h>\nextern "C" int slow(void) { usleep(300000); return 0; }\n')
    subprocess.run(["g++", "-shared", "-fPIC", str(src), "-o", str(so)], check=True)
    lib = P.load_library()
    names = ("paged_kv_write_rope", "paged_decode_attention_window", "paged_decode_step_window", "paged_prefill_attention_window")
    address = lambda fn: ctypes.cast(fn, ctypes.c_void_p).value
    P._native.set_functions(*[address(ctypes.CDLL(str(so)).slow)] * 4)
    yield P
    P._native.set_functions(*(address(getattr(lib, n)) for n in names))


def test_other_threads_run_during_a_call(slow_library):
    P = slow_library  # noqa: F811
    n, hq, hkv, d, bs = 2, 8, 2, 64, 16
    zeros = lambda *shape: torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    q, new, pool = zeros(n, 1, hq, d), zeros(n, 1, hkv, d), zeros(5, bs, hkv, d)
    tab, lens = torch.zeros((n, 2), dtype=torch.int32, device="cuda"), torch.ones(n, dtype=torch.int32, device="cuda")
    rope = P.Rope(64)
    attend = P.WindowDecodePlan(pool, pool, tab, lens, 0.1, hq, 8)
    step = P.WindowDecodePlan(pool, pool, tab, lens, 0.1, hq, 8, rope=rope)
    for call in (lambda: P.paged_kv_write_rope(q, new, new, rope, pool, pool, tab, lens), lambda: attend.run(q[:, 0]),
                 lambda: step.run(q[:, 0], new, new, lens), lambda: P.paged_prefill_attention_window(q, pool, pool, tab, lens, 0.1, 8)):
        t = threading.Thread(target=call)
        t0 = time.perf_counter()
        t.start()
        turns = 0
        while t.is_alive():
            time.sleep(0.001)
            turns += 1
        assert time.perf_counter() - t0 > 0.25               # the native call was made
        assert turns > 20, turns                             # and this thread ran meanwhile
