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
