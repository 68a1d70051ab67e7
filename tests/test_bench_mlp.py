"""bench.py --path mlp: its work model and its oracle arm (CPU), and a short run of the
training step against the layers' oracle (GPU)."""
import json
import os
import subprocess
import sys

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import bench  # noqa: E402
from newton_schulz_11_b200 import inputs  # noqa: E402


def test_blocks_of_the_workload():
    w = inputs.WORKLOADS[bench.MLP_WORKLOAD]
    layers = bench.mlp_layers(w)
    assert layers == [(1024, 4096)] * 24
    # six matrices a layer, the MLP's the last two
    assert len(bench.mlp_layers(w, 6)) == 1 and len(bench.mlp_layers(w, 12)) == 2


def test_work_model():
    products, ns = bench.mlp_work([(256, 1024)] * 2, 100, 5)
    # two matrices a block; each is used once forward and twice backward
    assert products == 2 * 2 * 3 * (2 * 100 * 256 * 1024)
    mw = bench.matrix_work(256, 1024)
    assert ns == 2 * 2 * 5 * (mw["gram"] + mw["poly"] + mw["apply"])


def test_oracle_arm_runs():
    w = inputs.WORKLOADS["single-256x128-f32"]
    ms, sample = bench.mlp_oracle_ms(w, [(64, 256)] * 3, 512, sample_tokens=32)
    assert ms > 0 and "3 blocks" in sample


@pytest.mark.gpu
def test_training_step_against_the_oracle():
    """Two blocks: the stack's input gradient and every gradient, then one optimizer step."""
    import torch

    from oracle import layers_oracle as lo

    assert torch.cuda.is_available(), "needs a B200"
    layers, tokens = [(128, 512)] * 2, 96
    step = bench.MlpTraining(layers, tokens, torch.device("cuda"), [(3.4445, -4.7750, 2.0315)] * 5)

    def f64(t):
        return t.detach().double().cpu().numpy()

    dx = f64(step.layers_pass())
    x, kept = f64(step.x), []
    for b in step.blocks:
        n, mean, rstd = lo.layer_norm(x, f64(b["gain"]), f64(b["beta"]))
        h, z = lo.linear(n, f64(b["w1"]), f64(b["b1"]), bench.MLP_ACT)
        kept.append((x, n, mean, rstd, h, z))
        x = lo.linear(h, f64(b["w2"]), f64(b["b2"]), "none", x)[0]
    dy, want = f64(step.dy), {}
    for i in (1, 0):
        b, (xi, n, mean, rstd, h, z) = step.blocks[i], kept[i]
        dz, want[i, "g_w2"], want[i, "g_b2"] = lo.linear_backward(dy, h, f64(b["w2"]), bench.MLP_ACT, z)
        dn, want[i, "g_w1"], want[i, "g_b1"] = lo.linear_backward(dz, n, f64(b["w1"]))
        dy, want[i, "g_gain"], want[i, "g_beta"] = lo.layer_norm_backward(dn, xi, mean, rstd, f64(b["gain"]), dy)
    # every tensor of the chain is rounded once to bf16, by half a step of 2^-8 of its value: at
    # most six in a row in a block, and the second block's on top of the first's
    tol = 2 * 6 * 2.0 ** -8
    assert np.linalg.norm(dx - dy) <= tol * np.linalg.norm(dy)
    for (i, name), ref in want.items():
        assert np.linalg.norm(f64(step.blocks[i][name]) - ref) <= tol * np.linalg.norm(ref), (i, name)
    before = [f64(b["w1"]) for b in step.blocks]
    step(torch.cuda.current_stream())
    torch.cuda.synchronize()
    for b, w0 in zip(step.blocks, before):
        assert np.isfinite(f64(b["w1"])).all() and not np.array_equal(f64(b["w1"]), w0)


@pytest.mark.gpu
def test_bench_line():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "bench.py"), "--path", "mlp", "--matrices", "12", "--steps",
                        "2", "--warmup", "3", "--no-cpu-baseline"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    line = json.loads(r.stdout.strip().splitlines()[-1])
    assert line["metric"] == "mlp_training_step_ms" and line["value"] > 0 and line["e2e"]["value"] > 0
    assert line["config"]["blocks"] == 2 and line["gpu_launches"] > 0
