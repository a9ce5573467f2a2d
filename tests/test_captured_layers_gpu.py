"""A plan's forward captured into a graph: every replay, between eager forwards
of the same plan, gives the forward of what x holds then."""

import dataclasses

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle  # noqa: E402
from synth import AdapterSpec, WorkloadSpec, make_workload  # noqa: E402

pytestmark = pytest.mark.gpu

ADAPTERS = [AdapterSpec("lora", rank=16, bias=True), AdapterSpec("dora", rank=16), AdapterSpec("oft", blk=32),
            AdapterSpec("vera"), AdapterSpec("ia3")]


@pytest.mark.parametrize("path", ["0", "1", "2", None])
@pytest.mark.parametrize("n, d_in, d_out", [(24, 512, 768), (128, 4096, 1024), (1000, 512, 640)])
def test_replays_match_what_x_holds(monkeypatch, path, n, d_in, d_out):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from lora_normal_form_amd import workload as glue
    if path is not None:
        monkeypatch.setenv("SCUTE_DECODE", path)
    rng = np.random.default_rng(n + d_in)
    wl = make_workload(WorkloadSpec("captured", "bf16", d_in, d_out, n, ADAPTERS, vera_rank=64, assign="explicit",
                                    token_adapter=rng.integers(-1, 5, n), seed=n))
    ld = glue.load(wl)
    xs = [ld.x * s for s in (1.0, -0.5, 2.0, 0.25, -3.0)]
    ld.layer.forward(ld.batch, ld.x, ld.W, ld.y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ld.layer.forward(ld.batch, ld.x, ld.W, ld.y, stream=torch.cuda.current_stream().cuda_stream)
    for step in range(8):
        x = xs[step % len(xs)]
        ld.x.copy_(x.roll(step, 0))
        ld.y.fill_(float("nan"))
        print(f"[gpu] path {path} n {n} step {step}", flush=True)
        if step in (2, 5):
            ld.layer.forward(ld.batch, ld.x, ld.W, ld.y)
        else:
            graph.replay()
        torch.cuda.synchronize()
        ref = oracle.forward(dataclasses.replace(wl, x=ld.x.cpu().double().numpy()))
        err = np.max(np.abs(ld.y.cpu().double().numpy() - ref)) / np.max(np.abs(ref))
        assert err <= 1e-2, (step, err)
    assert ld.batch.wait_failures() == 0
    ld.batch.close()
    ld.layer.close()


@pytest.mark.parametrize("adapters", [ADAPTERS, [AdapterSpec("ia3")]])
@pytest.mark.parametrize("path", ["0", "1", "2"])
@pytest.mark.parametrize("n", [24, 128, 700])
def test_launches_are_counted_and_timed(monkeypatch, path, n, adapters):
    """The cost's launches are those that are timed, before a plan's first capture
    and after it (a decode plan that counts or sums clears what it left first)."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from lora_normal_form_amd import scute
    from lora_normal_form_amd import workload as glue
    monkeypatch.setenv("SCUTE_DECODE", path)
    rng = np.random.default_rng(n)
    wl = make_workload(WorkloadSpec("counted", "bf16", 512, 768, n, adapters, vera_rank=64, assign="explicit",
                                    token_adapter=rng.integers(-1, len(adapters), n), seed=n))
    ld = glue.load(wl)
    handle = ld.layer.h

    def forward():
        scute.scute_profile_enable(handle, True)
        scute.scute_profile_read(handle)
        ld.layer.forward(ld.batch, ld.x, ld.W, ld.y)
        torch.cuda.synchronize()
        timed = scute.scute_profile_read(handle)
        scute.scute_profile_enable(handle, False)
        return sum(k["launches"] for k in timed.values()), ld.layer.cost(ld.batch)["launches"]

    timed, said = forward()
    assert timed == said
    y = ld.y.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ld.layer.forward(ld.batch, ld.x, ld.W, ld.y, stream=torch.cuda.current_stream().cuda_stream)
    after, said_after = forward()
    assert after == said_after, (timed, said, after, said_after)
    if path == "0" or n > 256 or len(adapters) > 1:  # (a two-launch plan without shrinks has nothing to clear)
        assert after - timed == (path != "0" and n <= 256), (timed, said, after, said_after)
    assert float((ld.y - y).abs().max()) <= 1e-2 * float(y.abs().max())
    ld.batch.close()
    ld.layer.close()
