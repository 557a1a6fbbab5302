"""The operators around the mixer in the debug build (libprism_debug.so, whose kernels check
their indices): on valid inputs it reports nothing and gives the release build's results bit
for bit.  The debug library is loaded in a child process, as in test_gpu_debug_bounds.py.
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _run_all():
    import linear_attention_sequence_shortconv_b200 as prism

    g = torch.Generator().manual_seed(9)

    def randn(*s, dtype=torch.float32):
        return torch.randn(s, generator=g).to(dtype).cuda()

    out = {}

    def keep(name, value):
        for i, t in enumerate(value):
            if t is not None:
                out[f"{name}_{i}"] = t.float().cpu().numpy()

    for dt in (torch.bfloat16, torch.float32):
        o, gate, w, dy = randn(3, 70, 2, 64, dtype=dt), randn(3, 70, 2, 64, dtype=dt), randn(64), randn(3, 70, 2, 64, dtype=dt)
        lens = torch.tensor([70, 0, 9], dtype=torch.int32).cuda()
        keep(f"gated_{dt}", [prism.gated_norm_fwd(o, gate, w, lengths=lens),
                             *prism.gated_norm_bwd(o, gate, w, dy, lengths=lens).values()])
        for D in (40, 77, 768, 2056):
            x, y, dh, dx = (randn(3, 70, D, dtype=dt) for _ in range(4))
            w, wp, s = randn(D), randn(D), randn(D)
            keep(f"block_{dt}_{D}", prism.block_norm_fwd(x, w, y=y, post_weight=wp, scale=s, lengths=lens))
            keep(f"block_bwd_{dt}_{D}", prism.block_norm_bwd(x, w, dh, y=y, post_weight=wp, scale=s, dx_out=dx,
                                                             lengths=lens).values())
    for n, V, D in ((500, 300, 96), (40000, 70000, 24), (3000, 2, 33)):
        ids = torch.randint(0, V, (1, n), generator=g).cuda()
        ids[0, : n // 2] = 1
        keep(f"embed_{n}", [prism.embed_fwd(ids, randn(V, D)), prism.embed_bwd(ids, randn(1, n, D), V)])
    for bits in (32, 8):
        p = [randn(n) for n in (1, 300, 5000)]
        state = prism.adamw_state(p, bits=bits)
        for step in (1, 2):
            prism.adamw_step(p, [randn(*t.shape) for t in p], step=step, **state)
        keep(f"adamw_{bits}", p + [t for x in state.values() for t in x])
    out["status"] = np.array(prism.stream_status())
    return out


def _child(path):
    import linear_attention_sequence_shortconv_b200 as prism

    assert prism.lib().prism_debug_bounds() == 1
    np.savez(path, **_run_all())


def test_debug_build_matches_release_and_reports_nothing(tmp_path):
    want = _run_all()
    path = str(tmp_path / "debug.npz")
    code = f"import tests.test_gpu_layer_debug as t; t._child({path!r})"
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, env=dict(os.environ, PRISM_DEBUG_BOUNDS="1"),
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-3000:]
    got = np.load(path)
    assert sorted(got.files) == sorted(want) and int(got["status"]) == 0 and int(want["status"]) == 0
    for name, value in want.items():
        assert np.array_equal(value, got[name]), name
