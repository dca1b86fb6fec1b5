"""Block operators on a stream that is not torch's current one, with inputs that the
caller drops as soon as the call returns."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU hosts
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import rope_rope3d_apply_gb300 as r  # noqa: E402

DEV = torch.device("cuda:0")
BF = torch.bfloat16


@pytest.mark.parametrize("tokens", [3, 500])
def test_temporaries_may_be_dropped_after_the_call(tokens):
    """The call waits behind a delay on its stream; its inputs' memory, free by then,
    is not what the current stream writes to meanwhile."""
    g = torch.Generator(device=DEV).manual_seed(tokens)
    normal = lambda *shape: (torch.randn(shape, generator=g, device=DEV) / shape[-1] ** 0.5).to(BF)  # noqa: E731
    x, y, w = normal(tokens, 512), normal(tokens, 512), (normal(1024, 512), normal(1024, 512), normal(512, 1024))
    calls = {
        "norm": lambda a, b, v, **k: r.rope3d_block_norm(a, b, post=r.NORM_RMS, **k),
        "norm backward": lambda a, b, v, **k: tuple(r.rope3d_block_norm_backward(a, b, a, b, post=r.NORM_RMS, **k).values()),
        "ffn": lambda a, b, v, **k: r.rope3d_gated_ffn(a, *v, keep=True, **k),
        "ffn backward": lambda a, b, v, **k: r.rope3d_gated_ffn_backward(b, a, *v, **k),
    }
    side = torch.cuda.Stream()
    for name, call in calls.items():
        want = call(x, y, w)
        torch.cuda.synchronize()
        a, b, v = x.clone(), y.clone(), tuple(t.clone() for t in w)
        sizes = [t.shape for t in (a, b, *v)]
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(100_000_000)
        out = call(a, b, v, stream=side)
        del a, b, v
        overwritten = [torch.full(s, -1.0, dtype=BF, device=DEV) for s in sizes]
        torch.cuda.synchronize()
        del overwritten
        assert all(torch.equal(p, q) for p, q in zip(out, want)), name


def test_captured_with_a_forked_stream():
    """Calls on a side stream, by the argument, inside a graph captured on another:
    temporaries dropped during the capture, replays with new inputs."""
    g = torch.Generator(device=DEV).manual_seed(5)
    normal = lambda *shape: (torch.randn(shape, generator=g, device=DEV) / shape[-1] ** 0.5).to(BF)  # noqa: E731
    x, dy, w = normal(200, 256), normal(200, 256), (normal(512, 256), normal(512, 256), normal(256, 512))

    def step(stream=None):
        _, n = r.rope3d_block_norm(x * 2.0, stream=stream)
        y, gp, up = r.rope3d_gated_ffn(n, *w, keep=True, stream=stream)
        return (y, *r.rope3d_gated_ffn_backward(dy, n, *w, gp, up, stream=stream))

    step()
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    doubled = torch.empty_like(x)
    with torch.cuda.graph(graph):
        torch.mul(x, 2.0, out=doubled)
        side.wait_stream(torch.cuda.current_stream())
        _, n = r.rope3d_block_norm(doubled, stream=side)
        y, gp, up = r.rope3d_gated_ffn(n, *w, keep=True, stream=side)
        out = (y, *r.rope3d_gated_ffn_backward(dy, n, *w, gp, up, stream=side))
        del n, y, gp, up
        torch.cuda.current_stream().wait_stream(side)
    for seed in (1, 2):
        x.copy_(torch.randn(x.shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, step()))
