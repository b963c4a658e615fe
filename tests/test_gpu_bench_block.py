"""bench.py --block-step: the training step around the layer is timed call by call beside the bench's
own line."""
import json
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
def test_block_step_is_timed_beside_the_line():
    print("[case] bench.py --config tiny --block-step", flush=True)
    r = subprocess.run([sys.executable, os.path.join(ROOT, "bench.py"), "--config", "tiny", "--steps", "3", "--warmup", "1",
                        "--cold-steps", "0", "--no-cpu-baseline", "--block-step"], capture_output=True, text=True, timeout=300,
                       cwd=ROOT)
    assert r.returncode == 0, r.stderr[-2000:]
    out = json.loads(r.stdout.strip())
    block = out["block_step"]
    assert block["ms_per_step"] > 0 and out["value"] > 0
    assert block["weights"] == 8 * 128 * 512 + 8 * 256 * 128 + 128 * 8 + 3 * 128
    assert all(v["ms"] > 0 for v in block["calls"].values())
    assert {"norm_before", "balance", "norm_behind", "balance_backward", "grad_norm", "adamw"} <= set(block["calls"])
