"""Expert routing called from several host threads at once, with sizes whose launches differ in
their shared memory and clusters. In child processes, so that the library's per-device setup is
part of what runs."""
import os
import subprocess
import sys
import textwrap

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# dynamic shared memory of 192, 33, 96 and 39 KB, clusters of 16, 16, 16 CTAs and 1
SETUP = textwrap.dedent(r"""
    import threading
    import torch
    from tests.oracle_helpers import gpu_ready
    m = gpu_ready()
    g = torch.Generator(device="cuda").manual_seed(3)
    sizes = [(30011, 2, 1024), (16384, 4, 16), (2100, 8, 512), (7, 3, 300)]
    ids = [torch.randint(-1, e, (t, k), generator=g, device="cuda") for t, k, e in sizes]
    torch.cuda.synchronize()
    errs = []
    gate = threading.Barrier(len(sizes))

    def run(work):
        def guarded(i):
            try:
                gate.wait()
                work(i)
            except Exception as e:  # reported below
                errs.append((sizes[i], repr(e)))
        ts = [threading.Thread(target=guarded, args=(i,)) for i in range(len(sizes))]
        for t in ts:
            t.start()
        for t in ts:
            t.join()
        assert not errs, errs
        assert m.device_status() == m.OK
""")

# The calls alone, one after another with next to nothing between, into buffers of each thread.
ROUTE = SETUP + textwrap.dedent(r"""
    streams = [torch.cuda.Stream() for _ in sizes]
    plans = [torch.zeros(e + 1 + t * k + m.route_rows(t, k, e), dtype=torch.int32, device="cuda")
             for t, k, e in sizes]
    torch.cuda.synchronize()

    def work(i):
        t, k, e = sizes[i]
        call, rows = m.lib().mxfp8_route, m.route_rows(t, k, e)
        at, stream = plans[i].data_ptr(), streams[i].cuda_stream
        args = (ids[i].data_ptr(), t, k, e, rows, at, at + 4 * (e + 1),
                at + 4 * (e + 1 + t * k), stream)
        got = [call(*args) for _ in range(4000)]
        streams[i].synchronize()
        bad = [s for s in got if s != m.OK]
        assert not bad, f"{len(bad)} of {len(got)} calls: status {bad[0]}"

    run(work)
    for i, (t, k, e) in enumerate(sizes):
        want = torch.cat([p.view(-1) for p in m.route(ids[i], e)])
        assert torch.equal(plans[i], want), sizes[i]
    print("THREADS_OK")
""")

# A layer's calls, through the package.
LAYER = SETUP + textwrap.dedent(r"""
    cols = 96
    ins = [(torch.randn(t, cols, generator=g, device="cuda").to(torch.bfloat16),
            torch.rand(t, k, generator=g, device="cuda")) for t, k, e in sizes]

    def layer(i, stream):
        (t, k, e), (x, w) = sizes[i], ins[i]
        kw = dict(stream=stream)
        plan = m.route(ids[i], e, **kw)
        y = m.dispatch(x, plan, w, **kw)
        act = m.swiglu(m.dispatch(x[:, :64].contiguous(), plan, **kw), **kw)
        return (*plan, y, *m.quantize_dispatch_dual(x, plan, w, **kw), m.combine(y, plan, w, **kw),
                *m.combine_backward(x, y, plan, w, **kw), *act,
                *m.swiglu_backward(act.h, act.codes, act.scales, recompute=True, **kw))

    outs = [None] * len(sizes)

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(20):
                outs[i] = layer(i, s)
        s.synchronize()

    torch.cuda.synchronize()
    run(work)
    for i in range(len(sizes)):
        for a, b in zip(outs[i], layer(i, None)):
            assert torch.equal(a, b), sizes[i]
    print("THREADS_OK")
""")

# Launches of two sizes in one graph, captured the larger first, and again the smaller first.
GRAPH = SETUP + textwrap.dedent(r"""
    for order in ((0, 3, 2), (3, 2, 0)):
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                held = [m.route(ids[i], sizes[i][2]) for i in order]
        m.route(ids[3], sizes[3][2])
        graph.replay()
        torch.cuda.synchronize()
        for i, plan in zip(order, held):
            for a, b in zip(plan, m.route(ids[i], sizes[i][2])):
                assert torch.equal(a, b), sizes[i]
    assert m.device_status() == m.OK
    print("THREADS_OK")
""")


@pytest.mark.parametrize("program", [ROUTE, LAYER, GRAPH], ids=["route", "layer", "graph"])
def test_sizes_do_not_disturb_one_another(program):
    r = subprocess.run([sys.executable, "-c", program], cwd=ROOT, env=dict(os.environ),
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "THREADS_OK" in r.stdout, \
        f"{r.stdout[-3000:]}\n{r.stderr[-3000:]}"
