"""muon_launch_count: what the library has queued, and the benchmark's figure from it."""
import json
import os
import subprocess
import sys

import pytest

from newton_schulz_11_b200 import _lib
from tests.conftest import cuda_present

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)


def test_refused_calls_are_not_counted():
    from newton_schulz_11_b200 import build

    build.build()
    if cuda_present():
        pytest.skip("other tests of this process launch kernels")
    lib = _lib.lib()
    before = lib.muon_launch_count()
    assert lib.muon_linear(None, None, 0, None) == _lib.MUON_ERR_INVALID_ARG
    assert lib.muon_layer_norm(None, None) == _lib.MUON_ERR_INVALID_ARG
    assert lib.muon_launch_count() == before == 0


@pytest.mark.gpu
def test_launches_are_counted():
    import ctypes

    import torch

    from newton_schulz_11_b200 import api

    lib = _lib.lib()

    def launched(call):
        before = lib.muon_launch_count()
        call()
        return lib.muon_launch_count() - before

    x, w = torch.randn(64, 128, device="cuda").bfloat16(), torch.randn(256, 128, device="cuda").bfloat16()
    _, mean, rstd = api.layer_norm(x)
    assert launched(lambda: api.layer_norm(x)) == 1
    assert launched(lambda: api.layer_norm_backward(x, x, mean, rstd)) == 2  # rows, and the join of their gradients
    assert launched(lambda: api.linear(x, w)) == 1
    assert launched(lambda: api.linear(x, w.float())) == 2  # the terms first
    assert launched(lambda: api.activation_backward(x, x, "gelu")) == 1
    assert launched(lambda: api.layer_norm(x[:0])) == 0
    p, g, m, v = ([torch.zeros(10, device="cuda") for _ in range(130)] for _ in range(4))
    assert launched(lambda: api.adamw_step(p, g, m, v, lr=0.1, step=1)) == 2  # 128 tensors a launch
    g, m = torch.randn(256, 128, device="cuda"), torch.zeros(256, 128, device="cuda")
    step = lambda: api.muon_step([w], [g], [m], lr=0.02)  # noqa: E731
    n = launched(step)
    _lib.check(lib.muon_profile_begin(), "muon_profile_begin")
    step()
    torch.cuda.synchronize()
    ms, count = (ctypes.c_double * 6)(), (ctypes.c_int64 * 6)()
    _lib.check(lib.muon_profile_end(ms, count, 6), "muon_profile_end")
    assert n == sum(count) > 10


@pytest.mark.gpu
def test_benchmark_reports_the_launches_of_its_steps():
    """The line of a run against the same training step here, counted."""
    import torch

    import bench
    from newton_schulz_11_b200 import inputs

    r = subprocess.run([sys.executable, os.path.join(ROOT, "bench.py"), "--path", "mlp", "--matrices", "12", "--steps",
                        "3", "--warmup", "3", "--no-cpu-baseline", "--no-e2e"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    line = json.loads(r.stdout.strip().splitlines()[-1])
    w = inputs.WORKLOADS[bench.MLP_WORKLOAD]
    step = bench.MlpTraining(bench.mlp_layers(w, 12), bench.MLP_TOKENS, torch.device("cuda"), bench.load_coeffs(w), lr=w.lr)
    lib = _lib.lib()
    before = lib.muon_launch_count()
    step(torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert line["gpu_launches"] == 3 * (lib.muon_launch_count() - before)


def test_source_hash_reads_files_only(tmp_path, monkeypatch):
    """A cache folder that a tool left among the sources does not end the benchmark."""
    import bench

    csrc = tmp_path / "newton_schulz_11_b200" / "csrc"
    csrc.mkdir(parents=True)
    (csrc / "a.cu").write_text("int a;")
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    h = bench.kernel_source_hash()
    (csrc / ".cache").mkdir()
    assert bench.kernel_source_hash() == h
