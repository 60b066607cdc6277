"""The scratch of sd_kv_attend: where it may begin, and who may use it at the same time."""

import pytest
import torch

import kvref
import verify_draft_prep_gb300 as sd

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Call:
    """Requests of uneven lengths, of which several CTAs share some."""

    def __init__(self, n_q, ctx, Hq, Hkv, D, seed):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        nb, self.table = kvref.make_table(ctx, 16, g, DEV)
        self.cache = kvref.make_cache(nb, 16, Hkv, D, g, DEV)
        n = sum(n_q)
        self.q = torch.randn(n, Hq, D, generator=g, device=DEV).bfloat16()
        self.cu = kvref.prefix(n_q, DEV)
        self.lens = torch.tensor(ctx, dtype=torch.int32, device=DEV)
        self.max_q = max(n_q)

    def __call__(self, out=None, **kw):
        out = torch.zeros_like(self.q) if out is None else out
        sd.sd_kv_attend(self.q, *self.cache, self.table, self.lens, self.cu, out, max_q=self.max_q,
                        **kw)
        return out


# units of 32, 64, 128 and 256 rows
FORMS = [(4, 8), (8, 8), (15, 8), (40, 8)]


@pytest.mark.parametrize("n,G", FORMS)
@pytest.mark.parametrize("D", [64, 128])
def test_scratch_at_any_multiple_of_16(n, G, D):
    c = Call([n, n, n], [9000, 200, 4000], 2 * G, 2, D, seed=n + D)
    need = sd.sd_kv_attend_workspace_bytes(D)
    room = torch.empty(need + 64, dtype=torch.uint8, device=DEV)
    want = c()
    for at in (0, 16, 32, 48):
        guard = torch.full((need + 64,), 0x5A, dtype=torch.uint8, device=DEV)
        room.copy_(guard)
        assert torch.equal(c(workspace_buf=room[at:at + need]), want)
        assert torch.equal(room[:at], guard[:at])
        assert torch.equal(room[at + need:], guard[at + need:])


def test_streams_without_scratch_of_their_own():
    """Calls whose requests are shared by many CTAs, on two streams at once: each as it is alone."""
    calls = [Call([40], [30000], 16, 2, 64, seed=1), Call([40], [28000], 16, 2, 64, seed=2),
             Call([30, 30], [9000, 15000], 16, 2, 128, seed=3)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    outs = [[torch.zeros_like(c.q) for _ in range(8)] for c in calls]
    torch.cuda.synchronize()
    for i in range(8):
        for j, (c, s) in enumerate(zip(calls, streams)):
            if i % 2:
                with torch.cuda.stream(s):
                    c(outs[j][i])
            else:
                c(outs[j][i], stream=s if i % 4 else s.cuda_stream)
    torch.cuda.synchronize()
    for w, got in zip(want, outs):
        for o in got:
            assert torch.equal(o, w)


def test_graphs_without_scratch_of_their_own():
    """Two graphs captured one after another, replayed together and beside an eager call."""
    calls = [Call([40], [30000], 16, 2, 64, seed=1), Call([60], [8000], 16, 2, 128, seed=2)]
    want = [c() for c in calls]
    outs = [torch.zeros_like(c.q) for c in calls]
    graphs = []
    for c, o in zip(calls, outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c(o)
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(4):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        eager = calls[0]()
        torch.cuda.synchronize()
        assert torch.equal(eager, want[0])
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
            o.zero_()
        torch.cuda.synchronize()


def test_refused_calls_give_their_scratch_back():
    """Head sizes and tensors that the call refuses, and calls without tokens."""
    c = Call([4], [100], 8, 2, 64, seed=4)
    c()
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for _ in range(3):
        with pytest.raises(sd.SDError):  # heads of 72 values
            sd.sd_kv_attend(torch.zeros(4, 8, 72, device=DEV).bfloat16(),
                            *(torch.zeros(8, 16, 2, 72, dtype=torch.uint8, device=DEV) for _ in range(2)),
                            *(torch.zeros(8, 2, device=DEV) for _ in range(2)), c.table, c.lens, c.cu,
                            torch.zeros(4, 8, 72, device=DEV).bfloat16())
        with pytest.raises(sd.SDError):  # more query heads than a multiple of the cache's
            sd.sd_kv_attend(c.q[:, :7], *c.cache, c.table, c.lens, c.cu, torch.zeros_like(c.q)[:, :7])
        with pytest.raises(sd.SDError):  # a tensor that the GPU cannot address
            sd.sd_kv_attend(c.q, *c.cache, c.table, c.lens.cpu(), c.cu, torch.zeros_like(c.q))
        sd.sd_kv_attend(c.q[:0], *c.cache, c.table, c.lens, c.cu, torch.zeros_like(c.q)[:0])
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() == before
