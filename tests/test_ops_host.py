"""Host code of the handle-less operators on the CPU: what two threads, or a failing CUDA call, can do to what is kept
between calls (the CUDA runtime's part is played by the tests)."""
import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "log_domain_sinkhorn_updates_b200", "csrc")

# Two threads ask for different shared-memory limits of one kernel at once.  The runtime's part: the limit is the last one
# set, and the call for the larger one is still under way when the other thread has its answer.
RUNTIME = r"""
#include <chrono>
#include <condition_variable>
#include <mutex>
static std::mutex mu;
static std::condition_variable cv;
int limit = 0, large_set = 0, small_done = 0;
void wait_for(int &flag) {
    std::unique_lock<std::mutex> l(mu);
    cv.wait_for(l, std::chrono::milliseconds(500), [&] { return flag != 0; });
}
void raise_flag(int &flag) {
    std::lock_guard<std::mutex> l(mu);
    flag = 1;
    cv.notify_all();
}
extern "C" {
int cudaGetDevice(int *d) { *d = 0; return 0; }
int cudaFuncSetAttribute(const void *, int, int bytes) {
    {
        std::lock_guard<std::mutex> l(mu);
        limit = bytes;
    }
    if (bytes == 200000) {
        raise_flag(large_set);
        wait_for(small_done);
    }
    return 0;
}
void **__cudaRegisterFatBinary(void *) { return nullptr; }
void __cudaRegisterFatBinaryEnd(void **) {}
void __cudaUnregisterFatBinary(void **) {}
char __cudaInitModule(void **) { return 0; }
}
"""
THREADS = r"""
#include <cstdio>
#include <thread>
#include "fs_ops.cuh"
extern int limit, large_set, small_done;
void wait_for(int &);
void raise_flag(int &);
void kernel() {}
int main() {
    std::thread large([] { fs::allow_smem<&kernel>(200000); });
    std::thread small([] {
        wait_for(large_set);
        fs::allow_smem<&kernel>(100000);
        raise_flag(small_done);
    });
    large.join();
    small.join();
    fs::allow_smem<&kernel>(200000);
    std::printf("limit %d\n", limit);
    return limit >= 200000 ? 0 : 1;
}
"""


def test_two_threads_on_first_use_leave_the_larger_shared_memory_limit(tmp_path):
    from log_domain_sinkhorn_updates_b200 import build
    if not shutil.which(build.NVCC):
        pytest.skip("no nvcc")
    (tmp_path / "runtime.cpp").write_text(RUNTIME)
    (tmp_path / "threads.cu").write_text(THREADS)
    subprocess.run([build.NVCC, "-std=c++17", "-cudart", "none", "-gencode", "arch=compute_100a,code=sm_100a", "-I", CSRC,
                    "-I", os.path.join(ROOT, "include"), "threads.cu", "runtime.cpp", "-o", "limits", "-lpthread"],
                   check=True, cwd=tmp_path)
    r = subprocess.run([str(tmp_path / "limits")], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout + r.stderr


def test_a_workspace_query_that_failed_is_not_kept(monkeypatch):
    """A geometry's first use while the device cannot be asked raises; its next one asks again."""
    import contextlib
    import types
    from log_domain_sinkhorn_updates_b200 import binding
    monkeypatch.setattr(binding, "_torch", types.SimpleNamespace(cuda=types.SimpleNamespace(
        device=lambda d: contextlib.nullcontext())))
    monkeypatch.setattr(binding, "_plans", {})
    answers = [ctypes.c_size_t(-1).value, 512, 1024]

    def plan():
        return binding._plan("geometry", lambda: (binding.FsAttnDesc(), "cuda:0"), lambda d: answers.pop(0))

    with pytest.raises(binding.FsError):
        plan()
    assert plan()[2] == 512 and plan()[2] == 512 and answers == [1024]


def test_workspace_queries_tell_a_failure_from_no_need():
    import torch
    if torch.cuda.is_available():
        pytest.skip("a device is present")
    from log_domain_sinkhorn_updates_b200 import binding, build
    build.build()
    L = binding.lib()
    view = binding.FsView(640, 64, 64)
    good = binding.FsAttnDesc(1, 10, 10, 1, 1, 64, 64, 1, 0.125, *[view] * 8)
    for grad in (0, 1):
        assert L.fs_cross_attn_workspace(ctypes.byref(good), grad) == ctypes.c_size_t(-1).value
        assert b"device" in L.fs_last_error(None).lower()
        xent = binding.FsXentDesc(5, 9, 64, 1, 1.0, 64, 64, 64, 64, -100)
        assert L.fs_cross_entropy_workspace(ctypes.byref(xent), None, None, grad) == ctypes.c_size_t(-1).value
        xent.v = 0
        assert L.fs_cross_entropy_workspace(ctypes.byref(xent), None, None, grad) == 0


@pytest.mark.parametrize("name", ["fs_cross_attn", "fs_cross_attn_grad", "fs_cross_entropy", "fs_cross_entropy_grad"])
def test_a_call_keeps_its_tensors(name):
    """No parameter is bound to anything else (an address, say) before the work is enqueued: Python hands the last reference
    of a temporary to the call, and the workspace could take the memory of one that the call let go."""
    import ast
    import inspect
    from log_domain_sinkhorn_updates_b200 import binding
    function = ast.parse(inspect.getsource(getattr(binding, name))).body[0]
    tensors = {a.arg for a in function.args.args} - {"scale", "ignore_index"}
    bound = {n.id for n in ast.walk(function) if isinstance(n, ast.Name) and isinstance(n.ctx, (ast.Store, ast.Del))}
    assert not tensors & bound
