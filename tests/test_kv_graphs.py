"""GPU checks of captured calls: every call of the cache on a stream that it names, the page calls over long lists
(their scratch in the graph), and two threads calling at once."""
import threading

import pytest
import torch

import _kv_ref as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def kv():
    import __graft_entry__
    __graft_entry__.build_library()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from attention_fa_fwd_02_gb300 import kv as m
    return m


def vec(*x):
    return torch.tensor(x, dtype=torch.int32).cuda()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_step_captured_on_a_named_stream(kv, dtype):
    """grow, append, attend, free of what was added: after each replay the cache is as it was, and O what a plain run
    gives for the replay's inputs."""
    cache = ref.make_cache(kv, [100, 37, 16], 16, 2, 64, dtype, extra=12, max_pages=20)
    rope = kv.Rope(64)
    new, slots = [2, 1, 30], vec(0, 1, 2)
    add, back, cu = vec(*new), vec(100, 37, 16), vec(0, 2, 3, 33)
    qkv = torch.zeros(33, 8 + 2 + 2, 64, dtype=dtype, device="cuda")
    out, lse = torch.empty(33, 8, 64, dtype=F32, device="cuda"), torch.empty(33, 8, device="cuda")
    s = torch.cuda.Stream()

    def step(stream):
        cache.grow(slots, add, stream=stream)
        q = cache.append(qkv[:, :8], qkv[:, 8:10], qkv[:, 10:], cu, slots, rope, stream=stream)
        cache.attend(q, cu, slots, out=out, lse=lse, stream=stream)
        cache.free(slots, back, stream=stream)

    step(None)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step(s)
    for i in range(4):
        qkv.copy_(torch.randn(qkv.shape, generator=torch.Generator().manual_seed(i)).to(dtype))
        graph.replay()
        got = out.clone(), lse.clone()
        out.fill_(7.0)
        step(None)
        assert torch.equal(got[0], out) and torch.equal(got[1], lse), i
        assert cache.lens.tolist() == [100, 37, 16]
    cache.check()


def test_the_page_calls_captured_over_long_lists(kv):
    n = 1300
    cache = kv.PagedCache.create(2, 6 * n, 8, 1, 16, n, 9)
    m = ref.Model(cache)
    g = torch.Generator().manual_seed(1)
    order = torch.randperm(n, generator=g).tolist()
    add = [(5 * i) % 23 for i in range(n)]
    src = [order[(i + 7) % n] for i in range(n)]
    some = order[::3] + [order[0], -1, n]
    keep = [(11 * i) % 19 for i in range(len(some))]
    args = [vec(*x) for x in (order, add, src, some, keep)]

    def calls():
        cache.grow(args[0], args[1])
        cache.fork(args[2], args[0])
        cache.free(args[3], args[4])
        cache.compact()

    def model():
        m.grow(order, add)
        m.fork(src, order)
        m.free(some, keep)
        m.compact()

    calls()
    model()
    m.same(cache, "as called")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for i in range(2):
        graph.replay()
        model()
        m.same(cache, i)


def test_two_threads_at_once(kv):
    caches = [ref.make_cache(kv, [4000 + 100 * i, 77], 16, 2, 64, BF, seed=i) for i in range(3)]
    qs = [torch.randn(2, 8, 64, generator=torch.Generator().manual_seed(i)).to(BF).cuda() for i in range(3)]
    cu = vec(0, 1, 2)
    want = [c.attend(q, cu) for c, q in zip(caches, qs)]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for k in range(200):
                    o, lse = caches[i].attend(qs[i], cu)
                    if k % 40 == 0:
                        s.synchronize()
                        if not (torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])):
                            wrong.append((i, k))
                s.synchronize()
        except Exception as e:  # (an exception of a thread would go unseen)
            wrong.append((i, e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
