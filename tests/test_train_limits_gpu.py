"""The cross entropy at its largest number of rows, against the definitions in fp32 on the GPU, a part of the rows at a time."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from consumer_gemm_chain_amd import MlpLoss  # noqa: E402

ROWS, H, V, PART = 1 << 24, 8, 10, 1 << 20


def test_loss_of_the_most_rows():
    """Eight products per logit and ten logits per row: fp32 errs by a few 2^-24 of values below 16, dz by 2^-11 of its unit,
    dx by 2^-11 of itself besides.  dw adds 2^24 rows: u |dz| |x| per row at random, of which ten times the root of the sum of
    squares is allowed, and for each of 2^24 / 32 steps of the accumulator 2^-24 of what it holds, which grows evenly to dw:
    eight times the root of their number times the largest.  With dloss left out (ones) most of dw is beyond fp16 and rounds
    to an infinity (from 65520 on)."""
    g = torch.Generator("cuda").manual_seed(5)
    x = torch.randn(ROWS, H, generator=g, device="cuda", dtype=torch.float16)
    w = torch.randn(V, H, generator=g, device="cuda").half()
    target = torch.randint(-2, V, (ROWS,), generator=g, device="cuda")
    loss, lse = torch.empty(ROWS, device="cuda"), torch.empty(ROWS, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    with MlpLoss(ROWS, H, V, "f16") as layer:
        layer.forward(x, w, target, loss, lse)
        layer.backward(x, w, target, lse, dx=dx, dw=dw)
        torch.cuda.synchronize()
    want, squares = (torch.zeros(V, H, device="cuda", dtype=torch.float64) for _ in range(2))
    w32 = w.float()
    for r in range(0, ROWS, PART):
        s = slice(r, r + PART)
        t, xs = target[s], x[s].float()
        z = xs @ w32.t().contiguous()
        counted = t >= 0
        rlse = torch.logsumexp(z, 1)
        rloss = rlse - z.gather(1, t.clamp(min=0)[:, None])[:, 0]
        for got, ref in ((lse[s], rlse), (loss[s], rloss)):
            assert float((got - torch.where(counted, ref, 0.0)).abs().max()) <= 2.0 ** -16
        dz = torch.softmax(z, 1)
        dz.scatter_add_(1, t.clamp(min=0)[:, None], torch.full((PART, 1), -1.0, device="cuda"))
        dz *= counted[:, None]
        ref = dz @ w32
        tol = 2.0 ** -11 * (ref.abs() + dz.abs() @ w32.abs()) + 2.0 ** -16 * w32.abs().sum()
        assert bool(((dx[s].float() - ref).abs() <= tol).all()), r
        d64, x64 = dz.double(), xs.double()
        want += d64.t().contiguous() @ x64
        squares += d64.square().t().contiguous() @ x64.square()
    tol = 2.0 ** -11 * want.abs() + 10 * 2.0 ** -11 * squares.sqrt() + 8 * (ROWS / 32) ** 0.5 * 2.0 ** -24 * want.abs().max()
    beyond = want.abs() - tol >= 65520
    assert bool((dw[beyond].double() == want[beyond].sign() * float("inf")).all())
    near = want.abs() + tol < 65504
    assert int(near.sum()) > 0 and bool(((dw.double() - want).abs() <= tol)[near].all())
