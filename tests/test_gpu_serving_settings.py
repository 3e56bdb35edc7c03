"""Attention over the 4-bit cache under the library's settings (fewer SMs, plain stream order) and beside other calls: two
streams with a workspace each, two captured graphs that share one and are replayed one after the other."""
import pytest

import serving_cases as C
from gpu_util import dev
from test_gpu_serving import attend, bf, check, expect, fg  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def few(d):
    return C.cache_case(d, [9000, 3, 17, 500], [2, 1, 0, 2], 8, 1, d, 32)


def many(d, hq):
    return C.wide(C.cache_case(d + hq, [900, 190, 40], [70, 80, 1], hq, 1, d, 16))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("sms", [1, 7, 60])
def test_on_fewer_sms(fg, d, sms):
    cases = [few(d), many(d, 8), many(d, 32)]
    assert [C.many_rows(c) for c in cases] == [False, True, True]
    fg.set_num_sms(sms)
    try:
        outs = [attend(fg, c) for c in cases]
        expect(fg)
    finally:
        fg.set_num_sms(0)
    for c, (out, ws) in zip(cases, outs):
        check(c, out)
        assert not ws[:7680].any(), "counters are left as they were"


def test_in_plain_stream_order(fg):
    was = fg.get_pdl()
    fg.set_pdl(False)
    try:
        cases = [few(128), many(128, 32)]
        outs = [attend(fg, c)[0] for c in cases]
    finally:
        fg.set_pdl(was)
    expect(fg)
    for c, out in zip(cases, outs):
        check(c, out)
        assert torch.equal(attend(fg, c)[0], out)


def arguments(c):
    return [bf(c["q_bits"])] + [dev(c[k]) for k in ("kc", "ks", "vc", "vs", "table", "start", "lens")]


@pytest.mark.parametrize("d", [64, 128, 256])
def test_two_streams_at_once(fg, d):
    cases = [few(d), many(d, 32)]
    args = [arguments(c) for c in cases]
    spaces = [fg.paged_attention_workspace(len(c["q"]), len(c["lens"]), c["hq"], c["hkv"], d) for c in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[torch.full_like(a[0], -77.0) for _ in range(12)] for a in args]
    torch.cuda.synchronize()
    for i in range(12):
        for a, ws, stream, out in zip(args, spaces, streams, outs):
            with torch.cuda.stream(stream):
                fg.paged_attention_mxfp4(*a, out[i], ws)
    torch.cuda.synchronize()
    expect(fg)
    for c, out in zip(cases, outs):
        check(c, out[0])
        assert all(torch.equal(out[0], x) for x in out[1:])


def test_two_graphs_share_a_workspace_in_turn(fg):
    cases = [few(128), many(128, 32)]
    args = [arguments(c) for c in cases]
    ws = fg.paged_attention_workspace(300, 1, 32, 1, 128)
    outs = [torch.full_like(a[0], -77.0) for a in args]
    graphs = []
    for a, out in zip(args, outs):
        fg.paged_attention_mxfp4(*a, out, ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            fg.paged_attention_mxfp4(*a, out, ws)
        graphs.append(graph)
    for _ in range(5):
        for out in outs:
            out.fill_(-77.0)
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for c, out in zip(cases, outs):
            check(c, out)
    expect(fg)
