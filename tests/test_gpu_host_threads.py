"""Calls from two host threads at once, each with its own stream, workspace and sizes. What a
launch sets up for its kernel belongs to the kernel on its device, not to the call: it must not
depend on the sizes, or one thread's sizes refuse the other's launch.

The threads are C threads (Python's take turns, so that two calls hardly ever meet)."""
import ctypes
import shutil
import subprocess

import pytest
import torch

from speculative_decoding_draft_sample_b200 import binding as bn

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16

SOURCE = r"""
#include <pthread.h>
#include <stddef.h>
typedef int (*norm_fn)(const void*, const void*, const void*, int, int, int, float, void*, void*, int, float*, float*,
                       void*, size_t, void*);
typedef int (*grad_fn)(const void*, const void*, const float*, const void*, const void*, int, int, int, void*, float*,
                       void*, size_t, void*);
typedef int (*sched_fn)(const float*, const float*, const float*, float, int, int, int, float, int*, float*, void*, size_t,
                        void*);
struct job {
  void* fn;
  int gradient, M, H, dtype, times, rc, failed;
  void *x, *weight, *y, *dx, *rstd, *ws, *stream;
  size_t bytes;
};
static void* loop(void* p) {
  struct job* j = (struct job*)p;
  for (int i = 0; i < j->times; ++i) {
    int rc = j->gradient ? ((grad_fn)j->fn)(j->x, j->weight, (float*)j->rstd, j->y, NULL, j->M, j->H, j->dtype, j->dx, NULL,
                                            j->ws, j->bytes, j->stream)
                         : ((norm_fn)j->fn)(j->x, NULL, j->weight, j->M, j->H, j->dtype, 1e-6f, NULL, j->y, j->dtype, NULL,
                                            (float*)j->rstd, j->ws, j->bytes, j->stream);
    if (rc != 0) {
      j->rc = rc;
      ++j->failed;
    }
  }
  return NULL;
}
static void* schedules(void* p) {  /* x: confidence logits, weight: position temperatures, rstd: step costs, y: cut, dx: survival */
  struct job* j = (struct job*)p;
  for (int i = 0; i < j->times; ++i) {
    int rc = ((sched_fn)j->fn)((float*)j->x, (float*)j->weight, (float*)j->rstd, 1.0f, j->M, j->H, 0, 0.0f, (int*)j->y,
                               (float*)j->dx, j->ws, j->bytes, j->stream);
    if (rc != 0) {
      j->rc = rc;
      ++j->failed;
    }
  }
  return NULL;
}
int run_at_once(struct job* jobs, int n) {
  pthread_t t[8];
  for (int i = 0; i < n; ++i)
    if (pthread_create(&t[i], NULL, jobs[i].gradient == 2 ? schedules : loop, &jobs[i])) return -1;
  for (int i = 0; i < n; ++i) pthread_join(t[i], NULL);
  return 0;
}
"""


class Job(ctypes.Structure):
    _fields_ = [("fn", ctypes.c_void_p)] + \
        [(k, ctypes.c_int) for k in ("gradient", "M", "H", "dtype", "times", "rc", "failed")] + \
        [(k, ctypes.c_void_p) for k in ("x", "weight", "y", "dx", "rstd", "ws", "stream")] + [("bytes", ctypes.c_size_t)]


@pytest.fixture(scope="module")
def runner(tmp_path_factory):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no C compiler")
    d = tmp_path_factory.mktemp("threads")
    (d / "threads.c").write_text(SOURCE)
    subprocess.run([gcc, "-O2", "-shared", "-fPIC", "-o", str(d / "threads.so"), str(d / "threads.c"), "-lpthread"], check=True)
    fn = ctypes.CDLL(str(d / "threads.so")).run_at_once
    fn.argtypes = [ctypes.POINTER(Job), ctypes.c_int]
    return fn


@pytest.mark.parametrize("gradient", [0, 1])
@pytest.mark.parametrize("dtype,widths", [(BF16, (1032, 4096)), (F32, (4104, 8192))])
def test_norms_of_two_widths(cuda_ok, runner, dtype, widths, gradient):
    """Both widths take the same kernel, with rings of different sizes."""
    M, name = 8, "dspark_residual_norm_grad" if gradient else "dspark_residual_norm"
    jobs, kept = (Job * 2)(), []
    for job, H in zip(jobs, widths):
        x = torch.randn(M, H, device="cuda").to(dtype)
        weight, ws = torch.ones(H, device="cuda", dtype=dtype), torch.zeros(bn.workspace_bytes(bn.OP_NORM, M, 0, H, 0, 0),
                                                                            dtype=torch.uint8, device="cuda")
        y, dx, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(M, device="cuda")
        bn.residual_norm(x, None, weight, 1e-6, y, ws, rstd=rstd)
        bn.residual_norm_grad(x, weight, rstd, y, dx, ws)
        stream = torch.cuda.Stream()
        kept.append((x, weight, ws, y, dx, rstd, stream, y.clone(), dx.clone()))
        job.fn = ctypes.cast(getattr(bn.lib(), name), ctypes.c_void_p).value
        job.gradient, job.M, job.H, job.dtype, job.times = gradient, M, H, bn._dtype_code(x), 20000
        job.x, job.weight, job.y, job.dx = x.data_ptr(), weight.data_ptr(), y.data_ptr(), dx.data_ptr()
        job.rstd, job.ws, job.stream, job.bytes = rstd.data_ptr(), ws.data_ptr(), stream.cuda_stream, ws.numel()
    torch.cuda.synchronize()
    assert runner(jobs, 2) == 0
    torch.cuda.synchronize()
    assert [(j.failed, j.rc) for j in jobs] == [(0, 0), (0, 0)]
    for k in kept:
        assert torch.equal(k[3], k[7]) and torch.equal(k[4], k[8])


def test_schedules_of_two_sizes(cuda_ok, runner):
    jobs, kept = (Job * 2)(), []
    for job, (B, K) in zip(jobs, [(64, 8), (1024, 8)]):
        conf, pos_temp = torch.randn(B, K, device="cuda"), torch.ones(K, device="cuda")
        cost = torch.arange(B * (K + 1), device="cuda", dtype=torch.float32) * 0.01
        cut, survival = torch.empty(B, device="cuda", dtype=torch.int32), torch.empty(B, K, device="cuda")
        ws = torch.zeros(bn.workspace_bytes(bn.OP_SCHEDULE, B, K, 8, 1, bn.F32), dtype=torch.uint8, device="cuda")
        bn.prefix_schedule(conf, pos_temp, cost, 1.0, bn.CUT_COST, 0.0, cut, survival, ws)
        stream = torch.cuda.Stream()
        kept.append((conf, pos_temp, cost, ws, stream, cut, survival, cut.clone(), survival.clone()))
        job.fn = ctypes.cast(bn.lib().dspark_prefix_schedule, ctypes.c_void_p).value
        job.gradient, job.M, job.H, job.times = 2, B, K, 5000
        job.x, job.weight, job.rstd, job.y, job.dx = (t.data_ptr() for t in (conf, pos_temp, cost, cut, survival))
        job.ws, job.stream, job.bytes = ws.data_ptr(), stream.cuda_stream, ws.numel()
    torch.cuda.synchronize()
    assert runner(jobs, 2) == 0
    torch.cuda.synchronize()
    assert [(j.failed, j.rc) for j in jobs] == [(0, 0), (0, 0)]
    for k in kept:
        assert torch.equal(k[5], k[7]) and torch.equal(k[6], k[8])
