"""GPU: the cached attention's workspace (few, long sequences) under calls on several streams at once."""
import pytest

from test_gpu_attention_views import b, dev, engines, make_cache, make_table, params, rows, run_cached, torch  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def long_request(engines):  # noqa: F811
    H, KV, D, page, held = 8, 2, 64, 64, 40000
    table, pages = make_table(200, [held], page)
    cache, p = make_cache(201, pages, KV, page, D), params(H, KV, D, dict(right=0))
    eng, q = engines["bf16"], [rows(202 + i, 2, H, D, "bf16") for i in range(2)]
    want = [run_cached(eng, x, cache, table, [held], [2], dict(right=0), D, max_len=held) for x in q]
    args = dev([0, 2]), dev([held]), dev(table), cache
    torch.cuda.synchronize()
    return eng, q, want, lambda x, out, stream: b.sf_attention_cached(eng, x, *args, out, p, max_len=held, stream=stream), \
        b.sf_attention_cached_workspace(eng, 2, 1, held, p)


def test_calls_on_two_streams_in_turn(long_request):
    """Calls on the current stream and on an explicit one with nothing between them: each has a workspace of its own."""
    eng, q, want, call, size = long_request
    assert size > 0
    side = torch.cuda.Stream()
    outs = [[torch.zeros_like(q[0]) for _ in range(40)] for _ in range(2)]
    torch.cuda.synchronize()
    for a, c in zip(*outs):
        call(q[0], a, None)
        call(q[1], c, side.cuda_stream)
    torch.cuda.synchronize()
    for got, w in zip(outs, want):
        assert all(torch.equal(o, w) for o in got)
    b.sf_check(eng)


@pytest.mark.parametrize("handle", ["stream", "default"])
def test_a_block_just_freed_is_left_to_its_readers(long_request, handle):
    """A tensor of the workspace's size, freed while its stream has still to write and read it, is not written by a call
    on another stream."""
    eng, q, want, call, size = long_request
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    out = torch.zeros_like(q[0])
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(other):
        x = torch.empty(size, dtype=torch.uint8, device="cuda")
        torch.cuda._sleep(20_000_000)   # about 10 ms
        x.fill_(77)
        y = x.clone()
        del x
        call(q[0], out, side.cuda_stream if handle == "stream" else 0)
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and (y == 77).all()
    b.sf_check(eng)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,n,H,KV,D", [(1, 1, 8, 8, 64), (2, 1, 16, 2, 128), (3, 2, 4, 1, 128), (1, 1, 32, 1, 64), (40, 1, 4, 4, 64)])
def test_a_workspace_for_any_length(engines, dt, T, n, H, KV, D):  # noqa: F811
    """The size for max_len 0 is enough for a call with max_len 0, of whatever table, and for every other."""
    eng, p = engines[dt], params(H, KV, D, {})
    most = b.sf_attention_cached_workspace(eng, T, n, 0, p)
    sizes = [b.sf_attention_cached_workspace(eng, T, n, x, p) for x in (1, 100, 4096, 8192, 10 ** 5, 10 ** 6, 2 ** 30)]
    assert sizes == sorted(sizes) and sizes[-1] == most
    if H * T <= 64:
        assert most > 0
    # the C call itself, with the documented 0 in both places
    held = 9000
    table, pages = make_table(205, [held] * n, 64)
    cache, q = make_cache(206, pages, KV, 64, D), rows(207, T, H, D, dt)
    new = [T // n + (i < T % n) for i in range(n)]
    want = run_cached(eng, q, cache, table, [held] * n, new, {}, D)
    cu = dev([sum(new[:i]) for i in range(n + 1)])
    args = dev([held] * n), dev(table), torch.full_like(q, 7.0), torch.empty(max(most, 1), dtype=torch.uint8, device="cuda")
    b._check(b.lib.sf_attention_cached(eng, q.data_ptr(), H * D, T, cu.data_ptr(), n, args[0].data_ptr(), args[1].data_ptr(),
                                       table.shape[1], 0, cache.desc, p, None, None, args[2].data_ptr(), H * D,
                                       args[3].data_ptr() if most else None, most, torch.cuda.current_stream().cuda_stream), eng)
    b.sf_check(eng)
    assert torch.equal(args[2], want)


@pytest.mark.parametrize("dt,D,rows_,tile,ctas", [("bf16", 64, 1, 8, 4), ("bf16", 64, 16, 16, 4), ("bf16", 128, 1, 8, 4),
                                                  ("bf16", 128, 16, 16, 3), ("f32", 64, 1, 8, 4), ("f32", 64, 16, 16, 3),
                                                  ("f32", 128, 1, 8, 3), ("f32", 128, 8, 8, 3)])
def test_a_split_stays_within_what_is_resident(engines, dt, D, rows_, tile, ctas):  # noqa: F811
    """One row tile over a very long past is split over as many clusters of 8 CTAs as its own kernel has resident at once
    (ctas: CTAs of an SM by its registers): clusters that wait for a second round cost more than they bring."""
    size = b.sf_attention_cached_workspace(engines[dt], 1, 1, 2 ** 30, b.attn_params(rows_, 1, D))
    clusters = size / ((rows_ // tile + 1) * tile * (D + 2) * 4)
    assert clusters == int(clusters)
    assert 2 <= clusters <= torch.cuda.get_device_properties(0).multi_processor_count * ctas // 8
