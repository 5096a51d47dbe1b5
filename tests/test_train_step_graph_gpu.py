"""A whole training step (block, norm, cross entropy, gradient norm, AdamW) captured once and replayed: each replay takes
the next step, bit for bit as eager calls do, with other batches, a schedule, and a step that is left out among them."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests.test_train_step_gpu import H, ROWS, V, Model  # noqa: E402


def states(m):
    o = m.opt
    return list(m.params) + list(o.master) + list(o.m) + list(o.v) + list(o.m_scale or []) + list(o.v_scale or []) + [o.t]


@pytest.mark.parametrize("dtype,act,bits", [("f16", "gelu_tanh", 8), ("bf16", "swiglu", 32)])
def test_whole_steps_replayed(dtype, act, bits):
    eager, graphed = Model(dtype, act, bits), Model(dtype, act, bits)
    gen = torch.Generator("cuda").manual_seed(5)
    x = torch.zeros(ROWS, H, dtype=eager.params[0].dtype, device="cuda")
    target = torch.zeros(ROWS, dtype=torch.int64, device="cuda")
    lr_scale = torch.ones(1, device="cuda")
    outs = {m: [torch.empty(1, device="cuda") for _ in range(2)] for m in (eager, graphed)}

    def step(m):
        norm, scale = outs[m]
        loss, grads = m.gradients(x, target)
        m.clip.forward(grads, norm, scale, max_norm=0.5, unscale=1 / m.scale_of_loss)
        m.opt.step(grads, 1e-2, scale=scale, lr_scale=lr_scale)
        return loss
    keep = [t.clone() for t in states(graphed)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(graphed)                       # (plans are made and the kernels are loaded before the capture)
    torch.cuda.synchronize()
    for t, k in zip(states(graphed), keep):
        t.copy_(k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step(graphed)
    for k in range(5):
        x.copy_(torch.randn(ROWS, H, generator=gen, device="cuda"))
        target.copy_(torch.randint(V, (ROWS,), generator=gen, device="cuda"))
        target[torch.rand(ROWS, generator=gen, device="cuda") < (0.0, 0.3, 0.99)[k % 3]] = -100
        lr_scale.fill_(0.5 ** k)
        if k == 3:
            x[5, 7] = float("inf")          # its gradients are not finite: the step is left out
        loss = step(eager)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(loss.view(torch.int32), captured.view(torch.int32)), k
        for a, b in zip(outs[eager], outs[graphed]):
            assert torch.equal(a.view(torch.int32), b.view(torch.int32)), k
        for a, b in zip(states(eager), states(graphed)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), k
    assert int(eager.opt.t) == 4
    del graph
    eager.close()
    graphed.close()
