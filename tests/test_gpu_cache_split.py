"""The split of an attention call over the CTAs, by itself: sizes whose attention would take minutes."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from gpu_util import require_gpu
from tree_forked_hybrid_gb300 import build as B

pytestmark = pytest.mark.gpu

C_STATUS, C_NITEM = 1, 6  # header words of a step's metadata


@pytest.fixture(scope="module")
def torch():
    return require_gpu()


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("probe") / "cache_split_probe.so")
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "cache_split_probe.cu")
    subprocess.run([B._nvcc(), *B.ARCH, "-O1", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr", "-shared", src,
                    "-o", so, "-lcudart_static", "-lrt", "-ldl", "-lpthread"], check=True, capture_output=True)
    L = ctypes.CDLL(so)
    L.probe_item_offset.restype = ctypes.c_int64
    return L


def split(torch, probe, caps, kt, Hkv, ctas):
    """(what each CTA found, the status word) for items of kt[i] tiles each."""
    T_cap, max_req, max_new, Hq, d = caps
    at = probe.probe_item_offset(T_cap, max_req, max_new, Hq, Hkv, d)
    meta = np.zeros(at + 8 * max(len(kt), 32), np.int32)  # (the first 32 records are read whatever the step holds)
    meta[C_NITEM] = len(kt)
    rec = meta[at:at + 8 * len(kt)].reshape(-1, 8)
    rec[:, 3], rec[:, 4] = 1, np.asarray(kt) * 128 - 1  # a new token behind the cached ones
    assert len(kt) <= T_cap // 8 + max_req  # (items of 8 tokens: the capacity holds them)
    m, out = torch.from_numpy(meta).cuda(), torch.full((ctas, 6), -9, dtype=torch.int64, device="cuda")
    assert probe.probe_split(ctypes.c_void_p(m.data_ptr()), T_cap, max_req, max_new, Hq, Hkv, d, ctas, ctypes.c_void_p(out.data_ptr())) == 0
    return out.cpu().numpy(), int(m[C_STATUS])


@pytest.mark.parametrize("n_item,lo,hi,Hkv,ctas", [
    (1, 1, 1, 1, 152), (1, 500, 500, 3, 152), (33, 1, 9, 8, 152), (5, 40, 300, 2, 148), (700, 1, 40, 4, 152),
    (131072, 16300, 16500, 1, 152),      # 2.1e9 tiles for a head, just past 2^31
    (131072, 21000, 33000, 1, 152), (131072, 8000, 9000, 4, 152), (150, 1 << 23, (1 << 24) - 1, 3, 256)])
def test_runs_cover_the_tiles(torch, probe, n_item, lo, hi, Hkv, ctas):
    kt = np.random.default_rng(n_item + lo).integers(lo, hi + 1, n_item)
    got, status = split(torch, probe, (1 << 20, 1024, 1 << 20, 32 * Hkv, 64), kt, Hkv, ctas)
    assert status == 0
    ends = np.cumsum(kt)  # 64 bits
    per_head = int(ends[-1])
    total = per_head * Hkv
    used = min(ctas, total)
    begin = 0
    for c in range(ctas):
        if c >= used:
            assert got[c, 0] == got[c, 1]
            continue
        n = total // used + (c < total % used)
        head, left = divmod(begin, per_head)
        item = int(np.searchsorted(ends, left, side="right"))
        off = left - (int(ends[item - 1]) if item else 0)
        assert got[c].tolist() == [begin, begin + n, head, item, off, c], c
        begin += n
    assert begin == total


def test_a_run_of_more_tiles_than_a_kernel_counts_is_refused(torch, probe):
    """More than 2^30 tiles for one CTA (attention of many minutes): no work, and the status says so."""
    got, status = split(torch, probe, (1 << 20, 1024, 1 << 20, 32, 64), np.full(131072, 1 << 21), 1, 152)
    assert status == 0x2 and bool((got[:, 0] == got[:, 1]).all())
