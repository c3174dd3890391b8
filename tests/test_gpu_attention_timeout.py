"""spec_verify_attention when its waits run out: builds of the library whose waits give up after 0, 700 and 2500 ns.  A call
returns, what no block reports SPEC_ST_TIMEOUT for is what the library itself computes, nothing is written out of place, and
the workspace serves the next call."""
import functools
import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

import numpy as np
import pytest
import torch

from speculative_decoding_verification_34_gb300 import build
from speculative_decoding_verification_34_gb300 import specverify as sv
from tests.test_gpu_attention import SENT, Case, dev

pytestmark = pytest.mark.gpu
LIMITS = (0, 700, 2500)


@pytest.fixture(scope="module")
def impatient(tmp_path_factory):
    """Limit in ns -> the library with that limit on a wait of the attention kernel."""
    build.build()
    rest = [os.path.join(build.BUILD, os.path.basename(s)[:-3] + ".o") for s in build.sources() if not s.endswith("attention.cu")]
    if not all(os.path.exists(o) for o in rest):
        build.build(force=True)
    out = tmp_path_factory.mktemp("impatient")

    def one(ns):
        obj, lib = str(out / f"attention{ns}.o"), str(out / f"lib{ns}.so")
        for cmd in ([build.nvcc(), *build.ARCH, *build.FLAGS, f"-DSPEC_ATTENTION_WAIT_NS={ns}", "-c",
                     os.path.join(build.CSRC, "attention.cu"), "-o", obj],
                    [build.nvcc(), *build.ARCH, "-shared", "-cudart", "static", "-o", lib, obj, *rest]):
            r = subprocess.run(cmd, capture_output=True, text=True)
            assert r.returncode == 0, r.stderr
        return lib

    with ThreadPoolExecutor(len(LIMITS)) as ex:
        return {ns: sv.load_library(p) for ns, p in zip(LIMITS, ex.map(one, LIMITS))}


@functools.cache
def case(name):
    rng = np.random.default_rng(50)
    if name == "batch":
        return Case(50, list(rng.integers(0, 3000, 60)), 4, 16, 4, 128, 32, num=rng.integers(0, 5, 60))
    if name == "trees":
        return Case(51, list(rng.integers(0, 900, 20)), 63, 8, 2, 128, 16, tree=True, num=rng.integers(20, 64, 20))
    if name == "shared":
        return Case(52, [30000, 40], 4, 4, 2, 64, 128)
    return Case(53, list(rng.integers(0, 50, 400)), 3, 4, 2, 64, 64)


@pytest.mark.parametrize("ns", LIMITS)
@pytest.mark.parametrize("name", ["batch", "trees", "shared", "short"])
def test_a_wait_that_runs_out_is_reported(monkeypatch, impatient, name, ns):
    c = case(name)
    ordinary = sv.load_library()
    need = sv.spec_attention_workspace_bytes(c.B, c.gmax, c.Hq, c.H, c.D)
    around = torch.full((need + 8192,), 0x5A, dtype=torch.uint8, device="cuda")
    ws = around[4096: 4096 + need]
    want, st = c.run(ws=ws)
    assert st == [0] * c.B
    size, guard = want.size, 4096
    flagged = 0
    for _ in range(6):
        flat = torch.full((size + 2 * guard,), SENT, dtype=torch.bfloat16, device="cuda")
        out = flat[guard: guard + size].view(want.shape)
        monkeypatch.setattr(sv, "_lib", impatient[ns])
        got, st = c.run(ws=ws, out=out)
        monkeypatch.setattr(sv, "_lib", ordinary)
        assert all(s in (0, sv.ST_TIMEOUT) for s in st)
        assert (flat[:guard] == SENT).all() and (flat[guard + size:] == SENT).all()
        assert (around[:4096] == 0x5A).all() and (around[4096 + need:] == 0x5A).all()
        for b, s in enumerate(st):
            rows = int(c.num[b]) + 1
            assert (got[b, rows:] == SENT).all(), b
            if s == 0:
                assert np.array_equal(got[b], want[b]), b
            else:
                flagged += 1
    assert flagged > 0 or ns > 0
    got, st = c.run(ws=ws)
    assert st == [0] * c.B and np.array_equal(got, want)


def test_a_call_without_status_words_returns(monkeypatch, impatient):
    c = case("batch")
    c.run()
    out, ws = torch.zeros_like(c.q).cuda(), sv.alloc_attention_workspace(c.B, c.gmax, c.Hq, c.H, c.D)
    monkeypatch.setattr(sv, "_lib", impatient[0])
    sv.spec_verify_attention(c.q.cuda(), c.gpu, dev(c.table), dev(c.lens), out, dev(c.num), workspace=ws)
    torch.cuda.synchronize()
