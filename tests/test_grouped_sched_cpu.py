"""CPU checks of the grouped products' scheduler (the code the kernel runs,
enumerated on the host): every output row and column of every group belongs
to exactly one tile, every tile's k-blocks to exactly one share, in range."""
import numpy as np
import pytest

from persistent_stream_matmul_gb300 import _binding as B
from persistent_stream_matmul_gb300 import build


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    B.load()


def _plan(kind, groups, rows, N, K, layout=1, sms=152, ctas=None):
    return B.GroupedPlan(kind, groups, rows, N, K, B.GEMM_BF16, layout, offline_sms=sms, ctas=ctas)


CASES = [([1], 8, 8), ([0, 1, 0], 64, 128), ([8] * 8, 1536, 2048), ([3, 0, 5, 1], 264, 520),
         ([1000, 0, 17, 256, 257, 255], 776, 200), ([0, 0], 64, 64), ([5000], 4096, 1024), ([2] * 300, 128, 4096),
         ([129, 3000, 1], 14336, 4096), ([0, 700, 0], 2048, 72), ([4000, 0, 70, 0], 256, 128), ([0, 5000, 3], 8, 8),
         ([3000, 40, 50, 0, 2000, 60, 70, 80, 1] * 4, 512, 640)]


@pytest.mark.parametrize("ctas", [1, 2])
@pytest.mark.parametrize("sms", [2, 20, 152])
@pytest.mark.parametrize("kind", [B.GEMM_GROUPED_ROWS, B.GEMM_GROUPED_INNER])
@pytest.mark.parametrize("counts,N,K", CASES)
def test_units_cover_every_tile_once(counts, N, K, kind, sms, ctas):
    offsets = np.concatenate([[0], np.cumsum(counts)])
    inner = kind == B.GEMM_GROUPED_INNER
    p = _plan(kind, len(counts), int(offsets[-1]) + 3, N, K, sms=sms, ctas=ctas)
    lanes, side = p.info("tile_m"), p.info("tile_n")
    m_total = K if inner else N  # col-major matrices: K is contiguous in C for INNER
    tiles = {}
    for u in range(p.info("units")):
        for tile, g, tm, n0, valid, width, k0, k1, kb in p.units(offsets, u):
            tiles.setdefault(tile, []).append((k0, k1, g, tm, n0, valid, width, kb))
            n = counts[g]
            assert kb == ((n if inner else K) + 63) // 64 and 0 <= k0 <= k1 <= kb and (k1 > k0 or (inner and n == 0))
            assert 0 < valid <= width <= side and width % (16 * ctas) == 0 and 0 <= tm * lanes < m_total
            if not inner:
                assert offsets[g] <= n0 and n0 + valid <= offsets[g + 1]
    split = [t for t in tiles if t < 0]
    units = sorted(-1 - t + i for t in split for i in range(len(tiles[t])))
    assert len(set(units)) == len(units) and (not units or units[-1] < p.info("units"))  # one share a unit
    assert all(len(tiles[t]) == 1 for t in tiles if t >= 0)
    covered = set()
    for shares in tiles.values():
        shares.sort()
        assert len({s[2:] for s in shares}) == 1
        kb = shares[0][7]
        at = 0
        for k0, k1, *_ in shares:
            assert k0 == at
            at = k1
        assert at == kb
        _, _, g, tm, n0, valid, _, _ = shares[0]
        for r in range(n0, n0 + valid):
            assert (g, tm, r) not in covered
            covered.add((g, tm, r))
    mt = -(-m_total // lanes)
    want = sum(N if inner else n for n in counts) * mt
    assert len(covered) == want
    p.close()


def test_shares_are_even_and_worth_joining():
    """Twelve column tiles of 128 k-blocks over 152 SMs: seven shares of at most
    twenty each, a unit each; with 32 k-blocks two; with 16 none."""
    for K, shares in ((8192, 7), (2048, 2), (1024, 1)):
        p = _plan(B.GEMM_GROUPED_ROWS, 64, 8, 1536, K)
        assert p.info("ctas") == 1 and p.info("units") == 152
        offsets = np.minimum(np.arange(65), 1)
        loads = [[k1 - k0 for *_, k0, k1, _ in p.units(offsets, u)] for u in range(152)]
        loads = [x for x in loads if x]
        assert all(len(x) == 1 for x in loads) and len(loads) == 12 * shares
        assert sum(x[0] for x in loads) == 12 * K // 64 and max(loads)[0] - min(loads)[0] <= 1
        p.close()


def test_a_remainder_of_tiles_is_split_first():
    """155 tiles of 64 k-blocks over 152 units: three tiles run first, in four
    shares each, then every unit has one whole tile."""
    p = _plan(B.GEMM_GROUPED_ROWS, 2, 128 * 155, 128, 4096, ctas=1)
    offsets = [0, 128 * 100, 128 * 155]
    work = [p.units(offsets, u) for u in range(152)]
    assert [len(x) for x in work] == [2] * 12 + [1] * 140
    assert all(w[0][7] - w[0][6] == 16 and w[0][0] == -1 - u // 4 * 4 for u, w in enumerate(work[:12]))
    assert all(w[-1][6:] == (0, 64, 64) for w in work)
    p.close()


def test_summed_rows_are_split_when_tiles_are_few():
    """One 256 x 256 gradient over 16384 rows: eleven shares of 23 or 24
    k-blocks."""
    p = _plan(B.GEMM_GROUPED_INNER, 1, 16384, 256, 256, ctas=2)
    loads = [sum(k1 - k0 for *_, k0, k1, _ in p.units([0, 16384], u)) for u in range(p.info("units"))]
    loads = [x for x in loads if x]
    assert len(loads) == 11 and set(loads) <= {23, 24} and sum(loads) == 256 and p.workspace_size > 0
    p.close()


def test_variant_rule_and_info():
    assert _plan(0, 8, 1024, 4096, 4096).info("ctas") == 1
    assert _plan(0, 8, 1025, 4096, 4096).info("ctas") == 2
    assert _plan(0, 1, 4096, 128, 4096).info("ctas") == 1
    assert _plan(0, 1, 4096, 512, 4096).info("ctas") == 1  # 32 tiles for 76 pairs
    assert _plan(0, 1, 8192, 512, 4096).info("ctas") == 2
    assert _plan(1, 8, 40, 256, 4096).info("ctas") == 2
    assert _plan(1, 4, 4096, 256, 4096).info("ctas") == 1  # 64 tiles for 76 pairs
    assert _plan(1, 8, 4096, 128, 4096).info("ctas") == 1
    p = _plan(0, 8, 4096, 4096, 4096)
    assert (p.info("tile_m"), p.info("tile_n"), p.info("units")) == (256, 256, 76)
    assert p.info("smem_bytes") <= 227 * 1024 and p.info("stages") >= 4 and p.workspace_size > 0
    p.set_option(B.GEMM_GROUPED_OPT_CTAS, 1)
    assert (p.info("tile_m"), p.info("units")) == (128, 152)
    for key, value, status in ((1, 3, B.GEMM_ERR_UNSUPPORTED), (1, -1, B.GEMM_ERR_UNSUPPORTED),
                               (2, 0, B.GEMM_ERR_INVALID_ARG)):
        with pytest.raises(B.GemmError) as e:
            p.set_option(key, value)
        assert e.value.status == status
    assert p.info("ctas") == 1
    with pytest.raises(B.GemmError):
        p.info(99)


def test_refusals_of_offline_plans():
    lib = B.load()
    for sms in (-1, 0, 1):
        with pytest.raises(B.GemmError) as e:
            _plan(0, 4, 8, 8, 8, sms=sms)
        assert e.value.status == B.GEMM_ERR_INVALID_ARG
    with pytest.raises(B.GemmError) as e:  # more tiles than an index holds
        _plan(0, 1024, 2 ** 31 - 1024, 2 ** 31 - 1024, 64)
    assert e.value.status == B.GEMM_ERR_UNSUPPORTED
    p = _plan(0, 4, 100, 64, 64)
    P = 0x1000
    assert lib.gemm_grouped_run(p.handle, P, P, P, P, P, None) == B.GEMM_ERR_NO_DEVICE
    assert lib.gemm_grouped_last_status(p.handle, None) == B.GEMM_ERR_NO_DEVICE
    assert lib.gemm_grouped_workspace_size(p.handle, None) == B.GEMM_ERR_INVALID_ARG
    for offsets in ([0, 10, 5, 20, 30], [0, 10, 20, 30, 101], [-1, 0, 0, 0, 0]):
        with pytest.raises(B.GemmError) as e:
            p.units(offsets, 0)
        assert e.value.status == B.GEMM_ERR_INVALID_ARG
    with pytest.raises(B.GemmError):
        p.units([0, 1, 2, 3, 4], p.info("units"))
