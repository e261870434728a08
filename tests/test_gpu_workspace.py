"""One workspace for calls after one another: of other numbers of query heads, of other caches, windowed and paged."""
import random

import pytest

from test_gpu_paged import _cache, _fill, _i32, _pages

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from bit_asymmetric_kv_02_b200 import kivi  # noqa: E402


def _workspace(nbytes):
    buffer = torch.zeros(nbytes + 256, dtype=torch.uint8, device="cuda")
    return buffer, buffer.data_ptr() + (-buffer.data_ptr()) % 256


def test_paged_and_windowed_calls_share_a_workspace():
    """Heads that many blocks share, so that parts and tickets are in use by every call."""
    g = torch.Generator("cuda").manual_seed(3)
    paged = _cache(num_pages=400, num_seqs=3, max_blocks=170, num_kv_heads=1)
    _fill(paged, g)
    lens = [20000, 9000, 300]
    _pages(paged, lens, random.Random(1))
    lens = _i32(lens)
    flat = kivi.KiviCache(2, 2, 8192, bits=4, num_q_heads=2)
    k, v = (torch.randn(2, 2, 7001, 128, generator=g, device="cuda").half() for _ in range(2))
    flat.prefill(k, v)
    calls = [("paged", hq, torch.randn(3, hq, 128, generator=g, device="cuda").half()) for hq in (1, 4, 8, 23, 64)]
    calls += [("window", hq, torch.randn(2, hq, 128, generator=g, device="cuda").half()) for hq in (2, 6, 16)]

    def size(kind, hq):
        return kivi.kivi_paged_workspace_bytes(paged.cfg, hq) if kind == "paged" else kivi.kivi_window_workspace_bytes(flat.cfg, hq)

    def call(kind, hq, q, ws, nbytes):
        out = torch.full_like(q, 9.0)
        s = torch.cuda.current_stream().cuda_stream
        if kind == "paged":
            kivi.kivi_paged_decode_attention(paged.cfg, paged.c, 3, lens.data_ptr(), None, q.data_ptr(), 3, hq, 0.1, 0, 0, out.data_ptr(),
                                             ws, nbytes, None, s)
        else:
            kivi.kivi_decode_attention_window(flat.cfg, flat.c, q.data_ptr(), hq, 0.1, 6500, 3, out.data_ptr(), ws, nbytes, None, s)
        return out

    wants = []
    for kind, hq, q in calls:
        buffer, ws = _workspace(size(kind, hq))
        wants.append(call(kind, hq, q, ws, size(kind, hq)))
        torch.cuda.synchronize()
    buffer, ws = _workspace(max(size(kind, hq) for kind, hq, _ in calls))
    order = list(range(len(calls))) * 3
    random.Random(2).shuffle(order)
    for i in order:
        kind, hq, q = calls[i]
        assert torch.equal(call(kind, hq, q, ws, buffer.numel() - 256), wants[i]), (kind, hq)


@pytest.mark.parametrize("bits", [2, 4])
def test_one_cache_with_several_numbers_of_query_heads(bits):
    """attend() of 2, 8 and 4 query heads on one cache's workspace, heads shared between warps."""
    g = torch.Generator("cuda").manual_seed(bits)
    k, v = (torch.randn(1, 2, 60000, 128, generator=g, device="cuda").half() for _ in range(2))

    def cache(heads):
        c = kivi.KiviCache(1, 2, 60032, bits=bits, num_q_heads=heads)
        c.prefill(k, v)
        return c

    qs = {h: torch.randn(1, h, 128, generator=g, device="cuda").half() for h in (2, 4, 8, 16)}
    wants = {h: cache(h).attend(q, out=torch.full_like(q, 9.0)) for h, q in qs.items()}
    one = cache(16)
    for h in (16, 2, 8, 4, 16, 4, 2, 8, 16):
        assert torch.equal(one.attend(qs[h], out=torch.full_like(qs[h], 9.0)), wants[h]), h
    for h in (16, 2, 8):
        out = torch.full_like(qs[h], 9.0)
        kivi.kivi_decode_attention_noalloc(one.cfg, one.c, qs[h].data_ptr(), h, 128 ** -0.5, out.data_ptr(), None,
                                           torch.cuda.current_stream().cuda_stream)
        assert torch.equal(out, wants[h]), h


def test_no_workspace_is_made_in_a_capture():
    """Of the stream that the call runs on, which need not be the current one."""
    cache = _cache(num_seqs=2)
    g = torch.Generator("cuda").manual_seed(1)
    _fill(cache, g)
    lens, q = _i32([40, 60]), torch.randn(2, 4, 128, generator=g, device="cuda").half()
    out, side, graph = torch.zeros_like(q), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        graph.capture_begin()
    with pytest.raises(RuntimeError, match="before the capture"):
        cache.attend(lens, q, out=out, stream=side)
    with torch.cuda.stream(side):
        graph.capture_end()
    assert not cache._ws
    cache.attend(lens, q, out=out)
    assert out.any() and cache.read_status() == 0
