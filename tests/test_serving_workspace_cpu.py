"""Workspace sizes of the serving operators: what a server allocates for its largest call has to
serve every smaller one.  No GPU."""
import pytest

from intra_spatial_pipelining_gb300 import build, sgp

CAPS = [1, 64, 127, 128, 129, 255, 256, 257, 500, 511, 512, 513, 1000, 1023, 1024, 1025, 1280, 1281,
        2048, 2049, 4097, 8192, 8193, 16384, 16385, 32768, 100000]


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return sgp.lib()


@pytest.mark.parametrize("nq,nkv", [(64, 8), (8, 1), (1, 1), (16, 1), (32, 4), (15, 3), (128, 8), (12, 12)])
def test_prefix_attention_workspace_grows_with_the_call(nq, nkv):
    d = sgp.make_heads(nq, nkv)
    size = sgp.sgp_prefix_attention_workspace_bytes
    for n in (0, 1, 7, 512):
        rows = [[size(d, T, cap, n) for T in range(1, 513)] for cap in CAPS]
        for cap, row in zip(CAPS, rows):                       # more sequences
            assert all(a <= b for a, b in zip(row, row[1:])), cap
        for a, b, ra, rb in zip(CAPS, CAPS[1:], rows, rows[1:]):   # longer caches
            assert all(x <= y for x, y in zip(ra, rb)), (a, b)
    for T in (1, 3, 64, 374, 375, 512):                        # more prefixes
        row = [size(d, T, 1024, n) for n in range(513)]
        assert all(a <= b for a, b in zip(row, row[1:])), T
    for T in (1, 64, 374, 512):                                # capacities one by one
        row = [size(d, T, cap, 1) for cap in range(1, 3000)]
        assert all(a <= b for a, b in zip(row, row[1:])), T


@pytest.mark.parametrize("G", [1, 3, 8, 16])
def test_prefix_attention_workspace_goes_by_the_group(G):
    """The own caches' partials: a chunk of 1024 positions leaves G rows of 64 + 2 floats."""
    d, rows = sgp.make_heads(8 * G, 8), 512 * 8 * 32 * G
    got = sgp.sgp_prefix_attention_workspace_bytes(d, 512, 32768, 0)
    assert rows * 66 * 4 <= got <= rows * 66 * 4 + 512 * 8 * 16 + 4096


def test_kv_evict_workspace_grows_with_the_call():
    size = sgp.sgp_kv_evict_workspace_bytes
    for nkv in (1, 3, 8):
        d = sgp.make_heads(nkv, nkv)
        row = [size(d, T, 4096) for T in range(1, 513)]
        assert all(a <= b for a, b in zip(row, row[1:]))
        row = [size(d, 64, b) for b in range(1, 5000)]
        assert all(a <= b for a, b in zip(row, row[1:]))
