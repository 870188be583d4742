"""GPU: chunk attention at the end of the longest cache the arguments allow (2^31 - 16 slots)."""
import math

import pytest

from tests import _cache as C
from tests._gpu import need_gpu, torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def X():
    need_gpu()
    from sparse_depth_token_gb300 import xmod
    xmod.load()
    return xmod


@pytest.mark.parametrize("after", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "fp32"])
def test_last_slots_of_the_longest_cache(X, kind, after):
    """A page of 8176 slots that stands 262656 times in the table, whose keys weigh nothing, and the last
    page: rows see it up to the fourth slot from its end, and NaN follow. after: the last row's own
    slot holds NaN too, which the rows before it do not see."""
    hd, P, pages = 32, 8176, 262657
    assert P * pages == 2 ** 31 - 16
    dtype = torch.float32 if kind == "fp32" else torch.bfloat16
    g = torch.Generator().manual_seed(5)
    k = torch.randn(2, 1, P, hd, generator=g)
    v = torch.randn(2, 1, P, hd, generator=g)
    n = 3
    q = torch.randn(n, hd, generator=g)
    q[:, 0] = 40.0
    k[1, :, :, 0] = 0.0
    k[0, :, :, 0] = -100.0              # scores 700 below: weights of 0
    handle = dict(k_scale=None, v_scale=None)
    if kind == "e4m3":
        k, v = k.to(torch.float8_e4m3fn), v.to(torch.float8_e4m3fn)
        for name in ("k_scale", "v_scale"):
            handle[name] = torch.ones(2, 1, P, device="cuda")
            handle[name][1, 0, P - 4:] = math.nan
        k.view(torch.uint8)[1, 0, P - 4:] = 0x7f
        v.view(torch.uint8)[1, 0, P - 4:] = 0x7f
    else:
        k[1, 0, P - 4:] = math.nan
        v[1, 0, P - 4:] = math.nan
        k, v = k.to(dtype), v.to(dtype)
    if after:
        v.view(torch.uint8 if kind == "e4m3" else v.dtype)[1, 0, P - 5] = 0x7f if kind == "e4m3" else math.nan
    k, v, q = k.cuda(), v.cuda(), q.cuda().to(dtype)
    table = torch.zeros(1, pages, dtype=torch.int32, device="cuda")
    table[0, -1] = 1
    cache = X.kv_cache(k, v, table, **handle)
    dm = C.dims(X, 1, 1, hd, "fp32" if kind == "fp32" else "bf16")
    o, lse = torch.full((n, hd), 7.0, device="cuda", dtype=dtype), torch.zeros(n, 1, device="cuda")
    ws = torch.zeros(X.cache_attention_chunk_workspace_bytes(dm, 1, n), dtype=torch.uint8, device="cuda")
    ints = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    X.cache_attention_chunk(dm, cache, q, ints([0, n]), None, ints([2 ** 31 - 20]), o, ws, lse=lse)
    assert X.sync_status(ws) == X.OK
    kd, vd = k[1, 0].double(), v[1, 0].double()
    if after:
        assert bool(torch.isnan(o[n - 1]).all())
    for m in range(n - 1 if after else n):
        seen = P - 4 - (n - 1 - m)
        z = kd[:seen] @ q[m].double() / math.sqrt(hd)
        w = torch.softmax(z, 0)
        ref, spread = w @ vd[:seen], w @ vd[:seen].abs()
        # scores: hd products in fp32; weights 2^-18 and their rounding to bf16 (e4m3 and bf16)
        size = float((kd[:seen].abs() @ q[m].double().abs()).max())
        rel = 2 * size * math.sqrt(hd) * 2.0 ** -24 + 2.0 ** -18 + (0.0 if kind == "fp32" else 2.0 ** -8)
        bound = spread * rel
        half = 2.0 ** -24 if kind == "fp32" else 2.0 ** -8
        err = (o[m].double() - ref).abs() - bound - half * (ref.abs() + bound)
        assert float(err.max()) <= 0, (m, float(err.max()))
        assert abs(float(lse[m]) - float(torch.logsumexp(z, 0))) <= rel + 1e-6 * abs(float(lse[m]))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_segments_that_take_longer_than_a_wait(X, kind):
    """Two chunks of one token for each SM, all of one sequence: 180 million slots and 64 by turns, so that
    every CTA works on a long segment, whose end another warp of it waits for with the next one's
    query, for longer than the limit of a wait without progress."""
    hd, P, pages = 32, 8176, 22016
    n = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    g = torch.Generator().manual_seed(6)
    k, v = (torch.randn(1, 1, P, hd, generator=g).cuda() for _ in range(2))
    if kind == "e4m3":
        k, v = k.to(torch.float8_e4m3fn), v.to(torch.float8_e4m3fn)
        scales = {name: torch.ones(1, 1, P, device="cuda") for name in ("k_scale", "v_scale")}
    else:
        k, v, scales = k.to(torch.bfloat16), v.to(torch.bfloat16), {}
    cache = X.kv_cache(k, v, torch.zeros(1, pages, dtype=torch.int32, device="cuda"), **scales)
    dm = C.dims(X, 1, 1, hd, "bf16")
    q = torch.randn(n, hd, generator=g).cuda().to(torch.bfloat16)
    o, lse = torch.zeros(n, hd, device="cuda", dtype=torch.bfloat16), torch.zeros(n, 1, device="cuda")
    ws = torch.zeros(X.cache_attention_chunk_workspace_bytes(dm, n, n), dtype=torch.uint8, device="cuda")
    start = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    lens = torch.tensor([P * pages, 64] * (n // 2), dtype=torch.int32, device="cuda")
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    X.cache_attention_chunk(dm, cache, q, start, torch.zeros(n, dtype=torch.int32, device="cuda"), lens, o, ws, lse=lse)
    end.record()
    assert X.sync_status(ws) == X.OK
    print("ms:", begin.elapsed_time(end))
    # the long sequence is one page 22016 times over: its softmax is that page's. fp32 sums of 2.8
    # million tiles: half a step, 2^-24, for each of them and of the four products of 16 keys, twice
    # that if they are cut off; the weights' and the output's rounding
    for rows, slots, times, adds in ((slice(0, n, 2), P, pages, 5 * P * pages / 64), (slice(1, n, 2), 64, 1, 5)):
        z = q[rows].double() @ k[0, 0, :slots].double().T / math.sqrt(hd)
        w, rel = torch.softmax(z, 1), adds * 2.0 ** -23 + 2.0 ** -16
        ref, spread = w @ v[0, 0, :slots].double(), w @ v[0, 0, :slots].double().abs()
        assert float(((o[rows].double() - ref).abs() - spread * (rel + 2.0 ** -7)).max()) <= 0
        assert float((lse[rows, 0].double() - torch.logsumexp(z, 1) - math.log(times)).abs().max()) <= math.log1p(rel)
