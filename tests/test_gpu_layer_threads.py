"""The layer operators from two host threads at once, each on a stream of its own, with calls of the same kernels that
need different amounts of shared memory: from Python, and from a C client whose threads no lock keeps apart."""
import os
import shutil
import subprocess
import threading

import pytest
import torch

from shot_allreduce_ranks_gb300 import build

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16
HERE = os.path.dirname(os.path.abspath(__file__))
CUDA = os.environ.get("CUDA_HOME", "/usr/local/cuda")


@pytest.fixture(scope="module")
def ar():
    build.build()
    import shot_allreduce_ranks_gb300
    return shot_allreduce_ranks_gb300


def normal(seed, *shape, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(BF16)


def norms(ar, cols):
    """The forward pass that copies rows ahead."""
    x, res, w = normal(1, 500, cols), normal(2, 500, cols), normal(3, cols)
    return lambda: ar.residual_norm(x, res, w)


def gradients(ar, cols):
    dy, dr, r, w = normal(4, 4, cols), normal(5, 4, cols), normal(6, 4, cols), normal(7, cols)
    return lambda: [t for t in ar.residual_norm_backward(dy, dr, None, r, w) if t is not None]


def experts(ar, tokens):
    t = [normal(8, tokens, 64), normal(9, tokens, 8), normal(10, 8, 32, 64, scale=0.1), normal(11, 8, 32, 64, scale=0.1),
         normal(12, 8, 64, 32, scale=0.2)]
    return lambda: [ar.moe_ffn(*t, 2)]


@pytest.mark.parametrize("make,sizes", [(norms, (8192, 1024)), (gradients, (8192, 6144)), (experts, (32, 1))])
def test_two_host_threads(ar, make, sizes):
    calls = [make(ar, n) for n in sizes]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    begin, failed = threading.Barrier(2), []

    def work(k):
        try:
            begin.wait(60)
            with torch.cuda.stream(torch.cuda.Stream()):
                for i in range(1000):
                    got = calls[k]()
                    if i % 100 == 0:
                        torch.cuda.current_stream().synchronize()
                        assert all(torch.equal(a, b) for a, b in zip(got, want[k])), "values"
                torch.cuda.current_stream().synchronize()
        except Exception as e:
            failed.append("thread %d: %r" % (k, e))

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


@pytest.fixture(scope="module")
def client(tmp_path_factory):
    if not shutil.which("gcc"):
        pytest.skip("gcc is not installed")
    build.build()
    exe = str(tmp_path_factory.mktemp("threads") / "layer_threads_client")
    pkg = os.path.dirname(build.LIB)
    cmd = ["gcc", "-std=gnu11", "-O2", "-Wall", "-Wextra", "-Werror", "-pthread", "-I", os.path.join(os.path.dirname(HERE), "include"),
           "-I", os.path.join(CUDA, "include"), os.path.join(HERE, "layer_threads_client.c"), "-L", pkg, "-l:" + os.path.basename(build.LIB),
           "-L", os.path.join(CUDA, "lib64"), "-lcudart", "-Wl,-rpath," + pkg, "-Wl,-rpath," + os.path.join(CUDA, "lib64"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return exe


@pytest.mark.parametrize("op", ["norm", "gradients", "experts"])
def test_two_threads_of_a_c_client(client, op):
    r = subprocess.run([client, op, "20000"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "40000 calls, 0 refused" in r.stdout
