"""The embedding, the router, the experts, the join and the cross entropy
together, as a language model's training step uses them."""
import gc
import importlib.util
import math
import os

import pytest
import torch

import zero_sharded_optimizer_flatten_gb300 as Z

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("sparse_lm_example", os.path.join(ROOT, "examples", "sparse_lm.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.fixture(autouse=True)
def _cuda_cleanup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    gc.collect()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def plain_forward(model, ids, targets, chosen, balance=1e-2, z=1e-3):
    """The example's model in 64 bits, with the experts that it chose."""
    def norm(v, w):
        return v / torch.sqrt(v.pow(2).mean(-1, keepdim=True) + 1e-6) * w

    ids, targets = ids.reshape(-1), targets.reshape(-1)
    kept = ids >= 0
    x = model.table[ids.clamp(min=0)] * math.sqrt(model.hidden) * kept[:, None]
    n = norm(x, model.w_pre[0])
    extra = 0.0
    for k, block in enumerate(model.blocks):
        s = n @ block.router.t()
        p = torch.softmax(s, -1)
        weights = p.gather(1, chosen[k])
        weights = weights / weights.sum(-1, keepdim=True)
        T, E = s.shape
        counts = torch.bincount(chosen[k].reshape(-1), minlength=E).double()
        extra = extra + balance * (counts * p.sum(0)).sum() * E / (block.topk * T * T)
        extra = extra + z * torch.logsumexp(s, 1).square().mean()
        every = torch.einsum("th,ehf->tef", n, block.w_in)
        every = torch.einsum("tef,efh->teh", torch.nn.functional.gelu(every), block.w_out)
        y = (weights[..., None] * every.gather(1, chosen[k][..., None].expand(*chosen[k].shape, n.shape[1]))).sum(1)
        x = x + model.scale * model.gate[k] * norm(y, model.w_post[k])
        n = norm(x, model.w_pre[k + 1])
    return torch.nn.functional.cross_entropy(n @ model.table.t(), targets, ignore_index=-1) + extra


def test_model_gradients_match_the_plain_model(monkeypatch):
    """In bf16: every product and join rounds at 2^-9, some twenty of them one
    after the other and 2^-9 sqrt(20) ~ 1e-2 for independent ones; a gradient is
    a sum of hundreds of such terms. 6e-2 of a parameter's largest gradient is
    beyond what these can add up to and far below what a wrong or missing term
    (a tied gradient left out, a balance loss without its share) would leave."""
    E = example()
    torch.manual_seed(1)
    model = E.SparseLM(vocab=300, hidden=64, inner=96, n_experts=4).to("cuda", torch.bfloat16)
    gen = torch.Generator(device="cuda").manual_seed(2)
    ids, targets = E.texts(300, 4, 40, gen)
    ids, targets = ids.clone(), targets.clone()
    ids[0, 30:] = -1          # a padded sequence
    targets[0, 29:] = -1
    chosen = []
    route = Z.expert_route

    def noted(*a, **k):
        out = route(*a, **k)
        chosen.append(out[0].long())
        return out
    monkeypatch.setattr(E.Z, "expert_route", noted)
    loss = model(ids, targets)
    loss.backward()
    exact = E.SparseLM(vocab=300, hidden=64, inner=96, n_experts=4).to("cuda", torch.float64)
    exact.load_state_dict({k: v.double() for k, v in model.state_dict().items()})
    ref = plain_forward(exact, ids, targets, chosen)
    ref.backward()
    assert abs(float(loss.detach()) - float(ref.detach())) <= 2e-2 * float(ref.detach())
    want = dict(exact.named_parameters())
    for name, p in model.named_parameters():
        g, r = p.grad.double(), want[name].grad
        assert float((g - r).abs().max()) <= 6e-2 * float(r.abs().max()), name
    # the table has both ends' gradients: a token that is never read and never a target has the head's alone
    assert float((model.table.grad.double() - want["table"].grad).norm()) <= 2e-2 * float(want["table"].grad.norm())


def test_tied_table_in_one_buffer():
    """The head's gradient, and the embedding's added to its rows, in one
    binary32 buffer, against autograd's sum."""
    g = torch.Generator(device="cuda").manual_seed(3)
    table = (torch.randn(400, 72, device="cuda", generator=g) / 8).to(torch.bfloat16).requires_grad_()
    ids = torch.randint(-1, 400, (150,), device="cuda", generator=g)
    targets = torch.randint(-1, 400, (150,), device="cuda", generator=g)
    x = Z.embedding(ids, table, scale=2.0)
    Z.linear_cross_entropy(x, table, targets).backward()
    ce = Z.zero_linear_cross_entropy(x.detach(), table.detach(), targets)
    dx, dw = Z.zero_linear_cross_entropy_backward(x.detach(), table.detach(), targets, ce,
                                                  torch.ones((), device="cuda"), dw_dtype=torch.float32)
    assert Z.zero_embedding_backward(dx, ids, 400, scale=2.0, out=dw, accumulate=True) is dw
    # the same terms; autograd's table rounds each end's to bf16 (2^-9) and their sum once more, the head's dz too
    size = float(dw.abs().max())
    assert float((table.grad.float() - dw).abs().max()) <= 4 * 2.0 ** -9 * size


def test_example_runs():
    history = example().train(steps=4, ranks=2, count=3, length=20, vocab=97, hidden=64, inner=64,
                              say=lambda *_: None)
    assert len(history) == 4 and all(math.isfinite(a) and math.isfinite(b) and b > 0 for a, b in history)


def test_step_captured_while_an_eager_graph_of_the_same_leaves_lives():
    """The calls that a training step makes, captured whole, while an eager
    autograd graph over the same table is alive: they go through the plain calls
    and leave autograd's nodes alone."""
    g = torch.Generator(device="cuda").manual_seed(4)
    table = (torch.randn(300, 64, device="cuda", generator=g) / 8).to(torch.bfloat16).requires_grad_()
    ids = torch.randint(0, 300, (90,), device="cuda", generator=g)
    targets = torch.randint(0, 300, (90,), device="cuda", generator=g)
    one = torch.ones((), device="cuda")
    alive = Z.linear_cross_entropy(Z.embedding(ids, table), table, targets)

    def step():
        t = table.detach()
        x = Z.zero_embedding(ids, t)
        ce = Z.zero_linear_cross_entropy(x, t, targets)
        dx, dw = Z.zero_linear_cross_entropy_backward(x, t, targets, ce, one)
        return ce.total, Z.zero_embedding_backward(dx, ids, 300, out=dw, accumulate=True)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        total, dw = step()
    graph.replay()
    want = step()
    assert torch.equal(total, want[0]) and torch.equal(dw, want[1])
    alive.backward()
    assert float(alive.detach()) == float(total[0])
