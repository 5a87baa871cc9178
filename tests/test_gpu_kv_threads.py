"""kv_attention from several host threads, on streams given to it and in graphs, without a workspace of the caller's:
the workspaces that the binding keeps are never written by two calls at once."""
import threading

import numpy as np
import pytest
import torch

import block_scaled_precision_mx_gb300 as mx
from tests.test_gpu_kv import attention_case, built, gpu  # noqa: F401

pytestmark = pytest.mark.gpu


def case(seed, lens, queries, heads=8, kv_heads=2):
    c = attention_case(np.random.RandomState(seed), lens, queries, heads, kv_heads, 128, 64, "bf16", 0)
    args = [c["q"], *(gpu(c[n]) for n in ("kc", "vc", "ks", "vs", "tables", "lens", "q_start"))]
    return args, max(queries)


def same(got, want):
    return all(torch.equal(g.view(torch.int16), w.view(torch.int16)) for g, w in zip(got, want))


def test_threads_on_one_stream():
    """Prompts (several launches a call, one with a planning kernel) and single tokens, all on one stream and one workspace."""
    cases = [case(1, [900, 40, 2000], [100, 40, 300]), case(2, [300, 1500], [300, 700]), case(3, [5000, 70, 3], [1, 1, 1]),
             case(4, [2500], [2500])]
    want = [mx.kv_attention(*args, most) for args, most in cases]
    torch.cuda.synchronize()
    wrong, errors, start = [], [], threading.Barrier(len(cases))

    def work(i):
        try:
            torch.cuda.set_device(0)
            args, most = cases[i]
            start.wait()
            for _ in range(8):
                got = [mx.kv_attention(*args, most) for _ in range(10)]
                wrong.extend((i, k) for k, g in enumerate(got) if not same(g, want[i]))
        except Exception as e:  # reported below, on the main thread
            errors.append((i, repr(e)))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    assert not wrong, wrong[:10]
    assert mx.mx_check() == mx.MX_OK


@pytest.mark.parametrize("lens,queries", [([3000, 75], [1, 1]), ([900, 400], [100, 400])])
@pytest.mark.parametrize("given", [False, True])
def test_graphs_and_calls_side_by_side(lens, queries, given):
    """A graph captured without a workspace, on torch's stream or forked to a stream that is passed in, replayed
    beside calls on both streams."""
    args, most = case(5, lens, queries)
    other, other_most = case(6, [700, 2000], [200, 1])
    want, other_want = mx.kv_attention(*args, most), mx.kv_attention(*other, other_most)
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    main, side, graph = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=main):
        if given:
            side.wait_stream(main)
        mx.kv_attention(*args, most, out=out, lse=lse, stream=side if given else None)
        if given:
            main.wait_stream(side)
    for _ in range(20):
        out.fill_(7)
        torch.cuda.synchronize()
        with torch.cuda.stream(main):
            graph.replay()
        with torch.cuda.stream(side):
            got = [mx.kv_attention(*other, other_most) for _ in range(2)]
        got += [mx.kv_attention(*other, other_most, stream=side)]
        got += [mx.kv_attention(*other, other_most)]
        torch.cuda.synchronize()
        assert same((out, lse), want)
        assert all(same(g, other_want) for g in got)
    assert mx.mx_check() == mx.MX_OK


def test_capture_of_a_stream_that_is_passed_in():
    """The captured stream is not torch's current one."""
    args, most = case(7, [900, 400], [100, 400])
    want = mx.kv_attention(*args, most)
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    side, graph, current = torch.cuda.Stream(), torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        with torch.cuda.stream(current):
            mx.kv_attention(*args, most, out=out, lse=lse, stream=side)
    for _ in range(3):
        out.fill_(7)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert same((out, lse), want)
    assert mx.mx_check() == mx.MX_OK
