"""The native marshalling gives up the interpreter's lock while the library is called, as ctypes does:
a launch may wait for room in the launch queue, and what makes room may need the lock."""
import ctypes
import shutil
import subprocess
import threading
import time

import pytest
import torch

from selective_state_space_56_b200 import ops

pytestmark = pytest.mark.gpu
DEV = "cuda"

# An entry point that waits (half a second at most) for another thread to set a flag.
STUB = r"""
#include <unistd.h>
volatile int flag = 0, seen = 0;
int stub(void) {
    for (int i = 0; i < 500 && !flag; ++i) usleep(1000);
    seen = flag;
    return 0;
}
"""


def test_other_threads_run_during_a_call(cuda_ok, tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("no C compiler")
    (tmp_path / "stub.c").write_text(STUB)
    subprocess.run(["gcc", "-shared", "-fPIC", "-O1", "-o", str(tmp_path / "stub.so"), str(tmp_path / "stub.c")],
                   check=True)
    so = ctypes.CDLL(str(tmp_path / "stub.so"))
    flag, seen = (ctypes.c_int.in_dll(so, n) for n in ("flag", "seen"))
    lib = ops.load_library()
    own = {n: ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in ops._native.names()}
    state, x = torch.ones(2, 8, device=DEV), torch.ones(2, 8, device=DEV)
    ready = threading.Event()

    def other():
        ready.set()
        time.sleep(0.05)
        flag.value = 1

    thread = threading.Thread(target=other)
    ops._native.bind(dict(own, mamba_gated_state_update=ctypes.cast(so.stub, ctypes.c_void_p).value))
    try:
        thread.start()
        ready.wait()
        ops.gated_state_update(state, x, x)
    finally:
        ops._native.bind(own)
    thread.join()
    assert seen.value == 1, "the other thread did not run before the call returned"
