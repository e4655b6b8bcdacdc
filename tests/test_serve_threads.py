"""Other Python threads while a serving call waits in the library (a stand-in for it: nothing is launched)."""
import ctypes
import shutil
import subprocess
import threading
import time

import pytest
import torch

import bit_weight_only_w4a16_gb300 as w4
from test_serve_launch_errors import NAMES, address, bound, calls  # noqa: F401

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(w4._fast is None, reason="built without the native binding")]


@pytest.mark.parametrize("name", NAMES)
def test_other_threads_run_while_a_call_waits(bound, tmp_path, name):  # noqa: F811
    """A launch may wait for room in its stream's queue, and what is queued may wait for a Python thread."""
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src, lib = tmp_path / "slow.c", tmp_path / "slow.so"
    src.write_text("#include <unistd.h>\nint slow(void) { usleep(400000); return 0; }\n")
    subprocess.run([cc, "-shared", "-fPIC", str(src), "-o", str(lib)], check=True)
    slow = ctypes.CDLL(str(lib)).slow
    call = calls()[name]
    call()
    torch.cuda.synchronize()
    ticks, stop = [], threading.Event()

    def tick():
        while not stop.is_set():
            ticks.append(time.monotonic())
            time.sleep(0.005)

    th = threading.Thread(target=tick)
    th.start()
    try:
        bound(slow)
        time.sleep(0.05)
        begin = time.monotonic()
        call()
        end = time.monotonic()
    finally:
        stop.set()
        th.join()
    assert end - begin > 0.35
    assert sum(begin < x < end for x in ticks) >= 5
