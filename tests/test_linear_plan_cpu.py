"""Which way a product of more than 64 rows takes, by the plan's host-only query: every way, and every kernel there is for
it, is taken by a size that the GPU tests run, whatever number of clusters a device of 152 SMs holds at once."""
import ctypes
import itertools
import os

import pytest

import speculative_decoding_verification_59_gb300 as sv

FEW, WHOLE, CLUSTERS, SHARES = sv.SPEC_MATMUL_FEW, sv.SPEC_MATMUL_WHOLE, sv.SPEC_MATMUL_CLUSTERS, sv.SPEC_MATMUL_SHARES
SMS = 152

# (way, a tile's weight rows, CTAs that take it together, parts of a tile): sizes that take it
WAYS = {
    (WHOLE, 64, 2, 1): [(100, 300, 400), (100, 700, 1024)], (WHOLE, 128, 2, 1): [(500, 3000, 400)], (WHOLE, 192, 2, 1): [(600, 4000, 528), (1100, 2600, 12288)],
    (WHOLE, 256, 2, 1): [(700, 5000, 528), (700, 5000, 1040)],
    (WHOLE, 64, 1, 1): [(300, 3000, 1040)], (WHOLE, 128, 1, 1): [(257, 5000, 1040)], (WHOLE, 192, 1, 1): [(600, 5000, 528)],
    (WHOLE, 256, 1, 1): [(300, 12000, 528)],
    (CLUSTERS, 64, 2, 2): [(128, 128, 2064)], (CLUSTERS, 64, 2, 4): [(128, 70, 8208)],
    (CLUSTERS, 128, 2, 2): [(250, 4000, 12304), (700, 1000, 16400), (600, 1000, 16384)],
    (CLUSTERS, 64, 1, 2): [(65, 3000, 2064)], (CLUSTERS, 64, 1, 4): [(100, 2000, 8208)], (CLUSTERS, 64, 1, 8): [(128, 64, 12304), (300, 128, 16384)],
}
# the same of shares; odd numbers of blocks among them, so that steps of two blocks begin and end anywhere
SHARED = {
    (64, 2): [(143, 5059, 14672), (195, 4992, 15872)], (64, 3): [(140, 2462, 20256), (138, 2766, 30960)], (64, 4): [(221, 1175, 32304)],
    (256, 2): [(2000, 3000, 8192), (642, 6540, 4448)], (256, 3): [(600, 2000, 16400)], (256, 5): [(148, 5292, 16288)],
}


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(sv.lib_path()):
        import __graft_entry__
        __graft_entry__.build()
    return sv.load_library()


@pytest.mark.parametrize("want,sizes", [(k, s) for k, v in WAYS.items() for s in v] +
                         [((SHARES, k[0], 2, k[1]), s) for k, v in SHARED.items() for s in v])
def test_way(want, sizes):
    # (38 clusters of four CTAs or 19 of eight would be every SM, which no device measured had: there (221, 1175, 32304)
    # takes clusters)
    for clusters in itertools.product((70, 74, 76), range(32, 38), range(14, 19)):
        way, W, together, groups, parts = sv.matmul_plan(*sizes, SMS, clusters)
        assert (way, W, together, parts) == want, (sizes, clusters)
        assert 0 < groups * together <= SMS or way == CLUSTERS


def test_few_rows():
    for M in (1, 16, 64):
        assert sv.matmul_plan(M, 4096, 4096, SMS) == (FEW, 128, 1, 0, 0)
    assert sv.matmul_plan(65, 4096, 4096, SMS)[0] != FEW


def test_refusals():
    good, clusters, plan = (65, 64, 128, SMS), (ctypes.c_int32 * 3)(76, 36, 16), (ctypes.c_int32 * 5)()
    call = sv.load_library().spec_matmul_plan
    assert call(*good, clusters, plan) == sv.SPEC_OK
    for i, v in ((0, 0), (1, -1), (2, 0), (3, -1), (0, 2147483647), (1, 2147483647), (2, 2147483647)):
        bad = list(good)
        bad[i] = v
        assert call(*bad, clusters, plan) == sv.SPEC_ERR_INVALID_ARG
    assert call(*good, None, plan) == sv.SPEC_ERR_INVALID_ARG and call(*good, clusters, None) == sv.SPEC_ERR_INVALID_ARG
    assert call(2000000000, 2000000000, 128, SMS, clusters, plan) == sv.SPEC_ERR_INVALID_ARG        # more tiles than 32 bits count
    with pytest.raises(sv.SpecVerifyError):
        sv.matmul_plan(0, 64, 64, SMS)
