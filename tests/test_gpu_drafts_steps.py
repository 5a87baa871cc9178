"""The operators for drafted tokens as a serving step uses them, one after the other over one cache, each held against the
64-bit reference on what the step has by then; and what surrounds such calls: guard bands around every output and
workspace, other streams, graphs, host threads."""
import threading

import numpy as np
import pytest
import torch

import block_scaled_precision_mx_gb300 as mx
from tests import drafts_reference as ref
from tests import kv_reference as kv
from tests.test_gpu_drafts import TYPES, f64, gpu, ok, probs, rotation, rows, starts
from tests.test_gpu_kv_guards import Guarded, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def cpu(t):
    return t.cpu().numpy()


@pytest.mark.parametrize("certain", [True, False])
@pytest.mark.parametrize("p,d,kv_heads,group,elem,kind", [(16, 64, 2, 2, mx.E5M2, "f16"), (64, 128, 1, 8, mx.E4M3, "bf16"),
                                                          (32, 128, 2, 3, mx.E4M3, "bf16")])
def test_drafting_steps(p, d, kv_heads, group, elem, kind, certain):
    """Requests that start with prompts and go on with trees; all but the last one's tokens stay or go as verification
    says, and every block is held once or free."""
    rng = np.random.RandomState(p + d + certain)
    dtype, half_step, smallest = TYPES[kind]
    requests, longest, vocab = 5, 400, 300
    blocks, width = 3 + requests * (longest // p), longest // p + 1
    tables = torch.full((requests, width), -1, dtype=torch.int32, device="cuda")
    free, free_count = torch.arange(blocks, dtype=torch.int32, device="cuda"), torch.full((1,), blocks, dtype=torch.int32, device="cuda")
    codes = [torch.zeros((blocks, kv_heads, p, d), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scale = [torch.zeros((blocks, kv_heads), device="cuda") for _ in range(2)]
    table = gpu(rotation(longest, d))
    qw, kw = (torch.from_numpy(1 + 0.3 * rng.randn(d)).to(dtype).cuda() for _ in range(2))
    lengths = torch.zeros(requests, dtype=torch.int32, device="cuda")
    kept_more = 0
    for step in range(7):
        # the prompts are chains, and all of their tokens stay; later steps have trees, and one request that rests
        nodes = rng.randint(1, 60, requests) if step == 0 else rng.randint(1, 40, requests)
        if step == 3:
            nodes[2] = 0
        q_start_host, t = starts(nodes), int(nodes.sum())
        after = lengths + gpu(nodes, torch.int32)
        q_start, slots, linear, info = mx.kv_block_tables(tables, lengths, after, free, free_count, t, p)
        assert np.array_equal(cpu(q_start), q_start_host) and int(info[1]) == 0
        parents = np.concatenate([ref.random_parents(rng, n, 1 if step == 0 else None) for n in nodes]).astype(np.int32)
        most, words = int(nodes.max()), -(-int(nodes.max()) // 64)
        mask, positions = mx.kv_draft_trees(gpu(parents), after, q_start, most)
        want = ref.trees(parents, cpu(after), q_start_host, words, 0, t)
        assert np.array_equal(cpu(mask).view(np.uint64), want[0]) and np.array_equal(cpu(positions), want[1])
        x = rows(rng, (t, (group + 2) * kv_heads, d), dtype, 0.3).cuda()
        q, k, v = x.split([group * kv_heads, kv_heads, kv_heads], dim=1)
        qn, kn = mx.qk_norm_rope(q, k, qw, kw, table, positions)
        for y, z, w in ((qn, q, qw), (kn, k, kw)):
            want, tol = ref.norm(f64(z), f64(w), cpu(table), cpu(positions), 1e-6, False, half_step, smallest)
            assert (np.abs(f64(y) - want) <= tol).all()
        before = [cpu(c) for c in codes], [cpu(s) for s in scale]
        mx.kv_cache_append(kn, v, slots, *codes, *scale, elem=elem)
        for i, z in enumerate((kn, v)):
            want = kv.append(f64(z), cpu(slots), before[0][i], before[1][i], elem)
            assert np.array_equal(cpu(codes[i]), want[0]) and np.array_equal(cpu(scale[i]), want[1])
        out, lse = mx.kv_tree_attention(qn, *codes, *scale, tables, after, q_start, most, mask, elem=elem)
        seen = ref.sees(cpu(mask).view(np.uint64), cpu(positions), cpu(after), q_start_host, 0)
        want, want_lse, tol, lse_tol = ref.tree_attention(f64(qn), *(cpu(c) for c in codes), *(cpu(s) for s in scale), cpu(tables),
                                                          cpu(after), q_start_host, seen, elem, d ** -0.5)
        assert (np.abs(f64(out) - want) <= tol + (np.abs(want) + tol) * half_step + smallest).all()
        assert (np.abs(f64(lse) - want_lse) <= lse_tol).all()
        # verification (of the prompts: nothing to verify, all stay)
        if step == 0:
            path, counts = gpu(np.concatenate([np.arange(n) for n in nodes]), torch.int32), gpu(nodes, torch.int32)
        else:
            target = probs(rng, t, vocab, 2.0)
            draft = None if certain else target
            drafts = np.full(t, -1, np.int32)
            for a, b in zip(q_start_host, q_start_host[1:]):
                for i in range(a + 1, b):  # likely ones, so that some stay
                    drafts[i] = rng.choice(vocab, p=target[a + parents[i]].astype(np.float64) / target[a + parents[i]].astype(np.float64).sum())
            accept, sample = rng.rand(t).astype(np.float32), rng.rand(requests).astype(np.float32)
            path, tokens, counts = mx.kv_verify_drafts(gpu(target), gpu(drafts), gpu(parents), q_start, gpu(accept), gpu(sample),
                                                       draft_probs=None if draft is None else gpu(draft))
            want = ref.verify(target, draft, drafts, parents, q_start_host, accept, sample)
            for g, w in zip((path, tokens, counts), want):
                assert np.array_equal(cpu(g), w)
            kept_more += int((cpu(counts) > 1).sum())
        before = [cpu(c) for c in codes], [cpu(s) for s in scale]
        kept = mx.kv_cache_compact(path, counts, after, q_start, tables, *codes, *scale, elem=elem)
        for i in range(2):
            want = ref.compact(cpu(path), cpu(counts), cpu(after), q_start_host, cpu(tables), before[0][i], before[1][i], elem)
            assert np.array_equal(cpu(codes[i]), want[0]) and np.array_equal(cpu(scale[i]), want[1])
            assert np.array_equal(cpu(kept), want[2])
        free_count = info[:1]
        free_count = mx.kv_block_tables(tables, after, kept, free, free_count, 0, p)[3][:1]
        lengths = kept
        held = [int(b) for r in range(requests) for b in cpu(tables)[r, :-(-int(cpu(lengths)[r]) // p)]]
        assert sorted(held + cpu(free)[:int(free_count)].tolist()) == list(range(blocks))
        ok()
    assert kept_more >= 2  # (a word on the inputs: some drafts stay)


# ------------------------------------------------------------------ what is written
@pytest.mark.parametrize("t,heads,kv_heads,d,rot", [(1, 1, 1, 64, 64), (37, 5, 2, 128, 64), (300, 3, 1, 80, 80), (9, 2, 2, 256, 32)])
def test_norm_writes_only_its_outputs(t, heads, kv_heads, d, rot):
    rng = np.random.RandomState(t)
    q, k = rows(rng, (t, heads, d), torch.bfloat16).cuda(), rows(rng, (t, kv_heads, d), torch.bfloat16).cuda()
    w = torch.ones(d, device="cuda", dtype=torch.bfloat16)
    table, positions = gpu(rotation(50, rot)), gpu(rng.randint(0, 50, t), torch.int32)
    out = {n: Guarded(x.shape, torch.bfloat16) for n, x in (("q", q), ("k", k))}
    mx.qk_norm_rope(q, k, w, w, table, positions, q_out=out["q"].t, k_out=out["k"].t)
    check(out, "qk_norm_rope")
    need = mx.load().qk_norm_rope_workspace_bytes(d)
    out = {"dq": Guarded(q.shape, torch.bfloat16), "dk": Guarded(k.shape, torch.bfloat16), "dqw": Guarded((d,), torch.float32),
           "dkw": Guarded((d,), torch.float32), "ws": Guarded((need,), torch.uint8)}
    mx.qk_norm_rope_backward(q, k, q, k, w, w, table, positions, dq=out["dq"].t, dk=out["dk"].t, dq_weight=out["dqw"].t,
                             dk_weight=out["dkw"].t, workspace=out["ws"].t)
    check(out, "qk_norm_rope_backward")


@pytest.mark.parametrize("nodes", [[1], [64, 0, 65, 33], [1024], [7] * 300])
def test_trees_verification_and_compaction_write_only_their_outputs(nodes):
    rng = np.random.RandomState(len(nodes))
    t, requests, vocab = int(sum(nodes)) + 3, len(nodes), 700
    parents = np.concatenate([ref.random_parents(rng, n) for n in nodes] + [np.zeros(3)]).astype(np.int32)
    q_start, lengths = gpu(starts(nodes)), gpu(np.array(nodes) + 20, torch.int32)
    most, words = max(nodes), -(-max(nodes) // 64)
    out = {"mask": Guarded((t, words), torch.int64), "positions": Guarded((t,), torch.int32)}
    mx.kv_draft_trees(gpu(parents), lengths, q_start, most, tree_mask=out["mask"].t, positions=out["positions"].t)
    check(out, "kv_draft_trees")
    target, drafts = gpu(probs(rng, t, vocab)), gpu(rng.randint(0, vocab, t), torch.int32)
    for draft in (None, target):
        out = {"path": Guarded((t,), torch.int32), "tokens": Guarded((t,), torch.int32), "counts": Guarded((requests,), torch.int32)}
        mx.kv_verify_drafts(target, drafts, gpu(parents), q_start, gpu(rng.rand(t).astype(np.float32)),
                            gpu(rng.rand(requests).astype(np.float32)), draft_probs=draft, path=out["path"].t,
                            tokens=out["tokens"].t, counts=out["counts"].t)
        check(out, "kv_verify_drafts")
    p, heads, d = 16, 3, 64
    held = -(-(np.array(nodes) + 20) // p)
    tables = np.full((requests, int(held.max())), -1, np.int32)
    order = rng.permutation(int(held.sum()))
    for r, h in enumerate(held):
        tables[r, :h] = order[int(held[:r].sum()):int(held[:r].sum()) + h]
    cache = (len(order), heads, p, d)
    out = {"kc": Guarded(cache, torch.uint8, gpu(rng.randint(0, 120, cache).astype(np.uint8))),
           "vc": Guarded(cache, torch.uint8, gpu(rng.randint(0, 120, cache).astype(np.uint8))),
           "ks": Guarded(cache[:2], torch.float32, gpu(2.0 ** rng.randint(-3, 4, cache[:2]).astype(np.float32))),
           "vs": Guarded(cache[:2], torch.float32, gpu(2.0 ** rng.randint(-3, 4, cache[:2]).astype(np.float32))),
           "kept": Guarded((requests,), torch.int32)}
    paths = [sorted(set([0] * (n > 0) + [i for i in range(n) if rng.rand() < 0.4])) for n in nodes]
    path = np.full(t, -1, np.int32)
    for r, way in enumerate(paths):
        path[starts(nodes)[r]:starts(nodes)[r] + len(way)] = way
    mx.kv_cache_compact(gpu(path), gpu(np.array([len(x) for x in paths], np.int32)), lengths, q_start, gpu(tables), out["kc"].t,
                        out["vc"].t, out["ks"].t, out["vs"].t, kept_lengths=out["kept"].t)
    check(out, "kv_cache_compact")


@pytest.mark.parametrize("d,kind,elem", [(64, "bf16", 0), (128, "f16", 1)])
@pytest.mark.parametrize("nodes", [3, 9, 30, 60, 130])
def test_tree_attention_writes_only_its_outputs(nodes, d, kind, elem):
    rng = np.random.RandomState(nodes + d)
    n, kv_heads, heads, p = np.array([nodes, 1, max(1, nodes // 2)]), 2, 8, 64
    lengths = n + np.array([5000, 0, 63])
    held = -(-lengths // p)
    tables = np.full((3, int(held.max())), -1, np.int32)
    for r, h in enumerate(held):
        tables[r, :h] = np.arange(int(held[:r].sum()), int(held[:r].sum()) + h)
    cache = (int(held.sum()), kv_heads, p, d)
    codes = [gpu(rng.randint(0, 100, cache).astype(np.uint8)) for _ in range(2)]
    scale = [torch.full(cache[:2], 2.0 ** -7, device="cuda") for _ in range(2)]
    t = int(n.sum()) + 2
    parents = gpu(np.concatenate([ref.random_parents(rng, int(x)) for x in n] + [np.zeros(2)]), torch.int32)
    q_start, lens = gpu(starts(n)), gpu(lengths, torch.int32)
    mask, positions = mx.kv_draft_trees(parents, lens, q_start, nodes)
    q = rows(rng, (t, heads, d), TYPES[kind][0], 0.2).cuda()
    need = mx.kv_attention_workspace_bytes(t, 3, nodes, heads, kv_heads, d)
    out = {"out": Guarded((t, heads, d), TYPES[kind][0]), "lse": Guarded((t, heads), torch.float32),
           "ws": Guarded((need,), torch.uint8, torch.zeros(need, dtype=torch.uint8))}
    for _ in range(2):
        mx.kv_tree_attention(q, *codes, *scale, gpu(tables), lens, q_start, nodes, mask, positions, elem=elem, window=3000,
                             out=out["out"].t, lse=out["lse"].t, workspace=out["ws"].t)
        check(out, "kv_tree_attention")
    assert (out["ws"].t[:4096] == 0).all()


# ------------------------------------------------------------------ other streams, graphs, threads
def calls():
    """The small operators on fixed inputs, as closures that give their outputs."""
    rng = np.random.RandomState(3)
    nodes = [5, 9, 0, 30]
    t = int(sum(nodes))
    parents = gpu(np.concatenate([ref.random_parents(rng, n) for n in nodes]), torch.int32)
    q_start, lengths = gpu(starts(nodes)), gpu(np.array(nodes) + 50, torch.int32)
    q, k = rows(rng, (t, 6, 128), torch.bfloat16).cuda(), rows(rng, (t, 2, 128), torch.bfloat16).cuda()
    w, table = torch.ones(128, device="cuda"), gpu(rotation(200, 128))
    _, positions = mx.kv_draft_trees(parents, lengths, q_start, 30)
    target, drafts = gpu(probs(rng, t, 5000)), gpu(rng.randint(0, 5000, t), torch.int32)
    accept, sample = gpu(rng.rand(t).astype(np.float32)), gpu(rng.rand(4).astype(np.float32))
    return [lambda **kw: mx.kv_draft_trees(parents, lengths, q_start, 30, **kw),
            lambda **kw: mx.qk_norm_rope(q, k, w, w, table, positions, **kw),
            lambda **kw: mx.qk_norm_rope_backward(q, k, k.new_ones(q.shape) + q, k + 1, w, w, table, positions, **kw),
            lambda **kw: mx.kv_verify_drafts(target, drafts, parents, q_start, accept, sample, draft_probs=target, **kw),
            lambda **kw: mx.kv_verify_drafts(target, drafts, parents, q_start, accept, sample, **kw)]


def test_other_streams_and_graphs():
    for call in calls():
        want = call()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = call(stream=side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        with torch.cuda.stream(side):
            got = call()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        graphs = []
        for _ in range(2):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                out = call()
            graphs.append((graph, out))
        for _ in range(3):
            for graph, out in graphs:
                for x in out:
                    x.zero_()
                graph.replay()
                call()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for _, out in graphs for a, b in zip(out, want))
    ok()


def test_host_threads():
    todo = calls()
    want = [c() for c in todo]
    torch.cuda.synchronize()
    wrong, errors = [], []

    def work(i):
        try:
            torch.cuda.set_device(0)
            for _ in range(30):
                if not all(torch.equal(a, b) for a, b in zip(todo[i % len(todo)](), want[i % len(todo)])):
                    wrong.append(i)
        except Exception as e:  # reported below, on the main thread
            errors.append(repr(e))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2 * len(todo))]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not errors and not wrong, (errors, wrong)
    ok()


def test_tensors_of_another_device_are_refused(monkeypatch):
    for call in calls():
        call()
        with monkeypatch.context() as m:  # (one GPU: as if another were the current one)
            m.setattr(torch.cuda, "current_device", lambda: 1)
            with pytest.raises(ValueError):
                call(stream=0)
    ok()
