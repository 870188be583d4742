"""GPU: chunks without keys among others, many to a CTA."""
import pytest

from tests import test_gpu_chunk as T
from tests._gpu import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def X():
    need_gpu()
    from sparse_depth_token_gb300 import xmod
    xmod.load()
    return xmod


@pytest.mark.parametrize("kind,some,none", [("bf16", 1, 4), ("bf16", 1, 6), ("bf16", 1, 8), ("bf16", 2, 3), ("bf16", 3, 17),
                                            ("e4m3", 1, 6), ("fp32", 1, 6)])
@pytest.mark.parametrize("hq,hkv,hd", [(48, 4, 128), (8, 4, 64), (4, 4, 32)])
def test_runs_of_segments_without_keys(X, kind, hq, hkv, hd, some, none):
    """Segments with keys, all of them masked, then as many without as a ring has stages, more or
    fewer: each is a tile that is there without a load."""
    shape = []
    while len(shape) * hkv < 152 * 2 * (some + none):
        shape += [(1 + (len(shape) + i) % 3, (30, 64, 2, 75)[(len(shape) + i) % 4]) for i in range(some)]
        shape += [(1 + i % 2, 0) for i in range(-(-none // hkv))]
    s = T._setup(X, kind, hq, hkv, hd, 16, shape)
    for _ in range(3):
        s["o"].fill_(-3)
        s["lse"].fill_(-3)
        T._call(s)
        assert X.sync_status(s["ws"]) == X.OK
    with_keys = [i for i, (_, n) in enumerate(shape) if n]
    for i in with_keys[:: max(1, len(with_keys) // 40)]:
        T._check_rows(s, i)
    for i, (n, slots) in enumerate(shape):
        if not slots:
            at = slice(s["first"][i], s["first"][i] + n)
            assert bool((s["o"][at] == 0).all()) and bool((s["lse"][at] == -float("inf")).all())


@pytest.mark.parametrize("kind", sorted(T.KINDS))
def test_ragged_chunks_some_without_keys(X, kind):
    """Thirty chunks of one to four hundred tokens, some of them longer than their sequences."""
    shape = [(45, 46), (37, 42), (79, 101), (294, 294), (19, 16), (0, 0), (1, 0), (4, 4), (3, 4), (391, 392), (34, 45), (5, 2),
             (87, 87), (5, 5), (127, 127), (166, 167), (111, 116), (260, 260), (39, 36), (3, 3), (388, 388), (8, 13), (51, 56),
             (0, 0), (15, 20), (60, 57), (13, 13), (3, 3), (364, 365), (26, 26)]
    s = T._setup(X, kind, 48, 4, 128, 128, shape, pad=8, lead=1, tail=1)
    T._call(s)
    T._check(s)
