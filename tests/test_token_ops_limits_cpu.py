"""Refusals at the ends of the integer ranges, on the host before any CUDA
call.  The addresses are made up, so these run only where no GPU could be
handed them."""
import glob

import numpy as np
import pytest

import newton_schulz_fp32_gb300 as nsg

pytestmark = pytest.mark.skipif(bool(glob.glob("/dev/nvidia[0-9]*")), reason="made-up addresses stay away from a GPU")

FAKE = 1 << 20
MOST = (1 << 63) - 1


@pytest.fixture(scope="module")
def lib():
    nsg.build()
    return nsg.lib()


def gradient(lib, param, parts=(), n=4096, accum_elems=1 << 20, workspace_bytes=1 << 24, overwrite=0, stride=None):
    p = np.array([param], dtype=nsg.PARAM_DTYPE)
    q = np.array(list(parts), dtype=nsg.PART_DTYPE)
    return lib.muon_embedding_grad(FAKE, accum_elems, FAKE, 0, stride or param[2], FAKE, 1, n, 1.0, overwrite,
                                   p.ctypes.data, q.ctypes.data if len(q) else None, len(q), FAKE, workspace_bytes,
                                   None)


@pytest.mark.parametrize("param,parts", [
    ((MOST - 100, 10, 64, 0, 0), []), ((MOST - 639, 10, 64, 0, 0), []), ((MOST, 1, 1, 0, 0), []),
    ((0, 10, 64, 0, 0), [(0, 640, MOST - 100)]), ((0, 10, 64, 0, 0), [(0, 300, 0), (300, 640, MOST - 339)]),
    ((MOST - 100, 10, 64, 0, 0), [(0, MOST, 0)])])
def test_a_parameter_that_ends_past_the_index_range_is_refused(lib, param, parts):
    """Its end must not wrap to a small number, which would be inside accum."""
    for overwrite in (0, 1):
        assert gradient(lib, param, parts, overwrite=overwrite) == nsg.MUON_ERR_INVALID
        assert "range" in lib.muon_last_error().decode() or "accum_elems" in lib.muon_last_error().decode()


@pytest.mark.parametrize("overwrite", [0, 1])
@pytest.mark.parametrize("n,cols", [(1 << 30, 1 << 17), (1 << 28, 1 << 20), (1 << 30, 1 << 30)])
def test_a_gradient_of_too_many_blocks_is_refused_before_anything_is_written(lib, overwrite, n, cols):
    """A grid past 2^31 - 1 blocks is known from the sizes, before the table is
    zeroed (overwrite) or the tokens are sorted."""
    rc = gradient(lib, (0, 1, cols, 0, 0), n=n, accum_elems=MOST, workspace_bytes=1 << 62, overwrite=overwrite)
    assert rc == nsg.MUON_ERR_UNSUPPORTED and "too many" in lib.muon_last_error().decode()
