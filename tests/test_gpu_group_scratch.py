"""The scratch of the UE8M0 per-group products beyond 128 rows: in stream
captures, beside them, and on many streams.  Every result has to be the bits of
the same call alone (test_gpu_gemm.py and test_gpu_linear_epilogue.py compare
those with the definitions)."""
import threading

import pytest
import torch

from gpu_util import lib

pytestmark = pytest.mark.gpu


class Product:
    """One product with weights of its own; run(out) on the current stream."""

    def __init__(self, m, n, k, seed, experts=0):
        F = lib()
        g = torch.Generator(device="cuda").manual_seed(seed)
        x = (torch.randn(m, k, generator=g, device="cuda") * 2.0 ** (seed % 7)).bfloat16()
        u8 = dict(dtype=torch.uint8, device="cuda")
        self.a, self.sa = torch.empty((m, k), **u8), torch.empty((k // 128, m), **u8)
        F.fp8_quantize_token_group(x, F.E4M3, F.SCALE_UE8M0, self.a, self.sa)
        rows = n * max(1, experts)
        w = torch.randn(rows, k, generator=g, device="cuda") * 2.0 ** -(seed % 5)
        self.b, self.sb = torch.empty((rows, k), **u8), torch.empty(((rows + 127) // 128, k // 128), **u8)
        F.fp8_quantize_block(w.bfloat16(), F.E4M3, F.SCALE_UE8M0, self.b, self.sb)
        self.experts = experts
        if experts:
            self.b, self.sb = self.b.view(experts, n, k), self.sb.view(experts, n // 128, k // 128)
            cuts = sorted(torch.randint(0, m, (experts - 1,)).tolist())
            self.offsets = torch.tensor([0] + cuts + [m], dtype=torch.int32, device="cuda")
        self.shape = (m, n)
        self.want = self.new()
        self.run(self.want)
        torch.cuda.synchronize()

    def new(self):
        return torch.zeros(self.shape, dtype=torch.bfloat16, device="cuda")

    def run(self, out):
        F = lib()
        if self.experts:
            F.fp8_gemm_group_experts(self.a, self.sa, self.b, self.sb, F.SCALE_UE8M0, self.offsets, out)
        else:
            F.fp8_gemm_group_epilogue(self.a, self.sa, self.b, self.sb, F.SCALE_UE8M0, out)


def captured(products, stream):
    outs = [p.new() for p in products]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        for p, o in zip(products, outs):
            p.run(o)
    return g, outs


@pytest.mark.parametrize("experts", [0, 4])
def test_capture_on_a_fresh_stream(experts):
    """No call before the capture has used its stream; a larger call follows a
    smaller one inside it, and the graph replays on another stream."""
    ps = [Product(m, 256, 512, i, experts) for i, m in enumerate((300, 700, 1500, 300))]
    g, outs = captured(ps, torch.cuda.Stream())
    assert all((o == 0).all() for o in outs)
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, p.want) for o, p in zip(outs, ps))
        for o in outs:
            o.zero_()


def test_larger_call_after_a_capture():
    """A later, larger call on the capture's stream grows that stream's buffer;
    the graph keeps its own."""
    st = torch.cuda.Stream()
    small, large = Product(300, 256, 512, 1), Product(5000, 2048, 1024, 2)
    with torch.cuda.stream(st):
        small.run(small.new())
    g, outs = captured([small], st)
    got = large.new()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        large.run(got)
    filler = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")  # memory given back
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], small.want) and torch.equal(got, large.want)
    del filler


def test_replays_beside_direct_calls():
    """Two graphs captured on one stream, replayed on two others at once, with
    direct calls on the capture's stream."""
    st, s1, s2 = (torch.cuda.Stream() for _ in range(3))
    ps = [Product(900, 640, 2048, i) for i in range(3)]
    g1, o1 = captured([ps[0]] * 2, st)
    g2, o2 = captured([ps[1]] * 2, st)
    o3 = [ps[2].new() for _ in range(60)]
    torch.cuda.synchronize()
    for o in o3:
        with torch.cuda.stream(s1):
            g1.replay()
        with torch.cuda.stream(s2):
            g2.replay()
        with torch.cuda.stream(st):
            ps[2].run(o)
    torch.cuda.synchronize()
    assert all(torch.equal(o, ps[0].want) for o in o1) and all(torch.equal(o, ps[1].want) for o in o2)
    assert all(torch.equal(o, ps[2].want) for o in o3)


def test_memory_goes_with_the_graph():
    """Graphs made and dropped one after another use one buffer between them."""
    p = Product(4096, 4096, 4096, 3)  # 1 MB of words
    st = torch.cuda.Stream()

    def cycle():
        g, outs = captured([p], st)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], p.want)

    cycle()
    before = torch.cuda.mem_get_info()[0]
    for _ in range(40):
        cycle()
    torch.cuda.synchronize()
    assert before - torch.cuda.mem_get_info()[0] < 24 << 20


def test_more_streams_than_buffers():
    """Streams beyond those with a buffer of their own."""
    ps = [Product(260 + 8 * i, 256, 1024, i) for i in range(4)]
    made = [torch.cuda.ExternalStream(h) for h in raw_streams(80)]
    outs = [p.new() for st in made for p in ps]
    torch.cuda.synchronize()
    for j, st in enumerate(made):
        with torch.cuda.stream(st):
            for i, p in enumerate(ps):
                p.run(outs[4 * j + i])
    torch.cuda.synchronize()
    assert all(torch.equal(o, ps[i % 4].want) for i, o in enumerate(outs))
    g, got = captured(ps, made[-1])
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, p.want) for o, p in zip(got, ps))


def raw_streams(count):
    """Handles of streams outside torch's pool (which hands out 32 in turn)."""
    import ctypes
    rt = ctypes.CDLL("libcudart.so.13")
    out = []
    for _ in range(count):
        h = ctypes.c_void_p()
        assert rt.cudaStreamCreateWithFlags(ctypes.byref(h), 1) == 0
        out.append(h.value)
    return out


def test_threads_on_one_stream():
    """Calls of two threads on one stream do not take each other's words."""
    ps = [Product(400, 384, 1024, i) for i in range(2)]
    outs = [[p.new() for _ in range(200)] for p in ps]
    torch.cuda.synchronize()

    def work(i):
        for o in outs[i]:
            ps[i].run(o)

    ts = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    torch.cuda.synchronize()
    for p, os_ in zip(ps, outs):
        assert all(torch.equal(o, p.want) for o in os_)
