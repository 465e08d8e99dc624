"""The training-step operators together, and the engine's gradient clipping."""
import gc
import importlib.util
import math
import os

import pytest
import torch

import zero_sharded_optimizer_flatten_gb300 as Z
from zero_sharded_optimizer_flatten_gb300.engine import ZeroEngine

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location(
        "sparse_block_example", os.path.join(ROOT, "examples", "sparse_block.py"))
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


def plain_forward(model, tokens):
    """The example's model in 64 bits, experts chosen for every token at once."""
    def norm(v, w):
        return v / torch.sqrt(v.pow(2).mean(-1, keepdim=True) + 1e-6) * w

    x = tokens @ model.lift.weight.t() + model.lift.bias
    n = norm(x, model.w_pre[0])
    for k, block in enumerate(model.blocks):
        score = torch.softmax(n @ block.router.t(), dim=-1)
        weights, ids = score.topk(block.topk, dim=-1)
        weights = weights / weights.sum(dim=-1, keepdim=True)
        every = torch.einsum("th,ehf->tef", n, block.w_in)
        every = torch.einsum("tef,efh->teh", torch.nn.functional.gelu(every), block.w_out)
        y = (weights[..., None] * every.gather(1, ids[..., None].expand(*ids.shape, n.shape[1]))).sum(1)
        x = x + model.scale * model.gate[k] * norm(y, model.w_post[k])
        n = norm(x, model.w_pre[k + 1])
    return n @ model.head.weight.t() + model.head.bias


def test_model_gradients_match_the_plain_model():
    """In fp32 throughout: the model's own products round at 2^-11 at worst
    (tf32 off: 2^-24), the sums are short, so outputs and gradients agree to
    1e-4 of their size."""
    E = example()
    torch.manual_seed(3)
    model = E.SparseModel(width=24, hidden=96, inner=64, out=5, n_experts=6).to("cuda")
    with torch.no_grad():
        for p in list(model.w_pre) + list(model.w_post) + list(model.gate):
            p.add_(0.1 * torch.randn_like(p))
    tokens = torch.randn(64, 24, device="cuda")
    out = model(tokens)
    c = torch.randn_like(out)
    (out * c).sum().backward()
    got = {k: p.grad.clone() for k, p in model.named_parameters()}
    wide = E.SparseModel(width=24, hidden=96, inner=64, out=5, n_experts=6).to("cuda", torch.float64)
    wide.load_state_dict({k: v.double() for k, v in model.state_dict().items()})
    ref = plain_forward(wide, tokens.double())
    (ref * c.double()).sum().backward()
    assert float((out - ref).detach().norm()) <= 1e-4 * float(ref.detach().norm())
    for k, p in wide.named_parameters():
        assert float((got[k] - p.grad).norm()) <= 1e-4 * float(p.grad.norm()) + 1e-7, k


def test_example_trains():
    history = example().train(steps=40, say=lambda *_: None)
    first = sum(h[0] for h in history[:5]) / 5
    last = sum(h[0] for h in history[-5:]) / 5
    assert last < 0.6 * first
    assert all(math.isfinite(h[1]) and h[1] > 0 for h in history)


@pytest.mark.parametrize("offload", [None, "host_state", "cpu"])
@pytest.mark.parametrize("mode", ["flat", "round_robin"])
def test_engine_clips_the_reduced_gradient(offload, mode):
    """clip_grad_norm takes the norm over all shards and scales them; the
    step then uses them.  A second engine without clipping, fed gradients
    that are small enough, is left as it was."""
    def engine():
        torch.manual_seed(5)
        net = torch.nn.Sequential(torch.nn.Linear(37, 61), torch.nn.Tanh(),
                                  torch.nn.Linear(61, 3)).to("cuda", torch.bfloat16)
        return net, ZeroEngine(net.parameters(), 3, mode=mode, offload=offload)

    def backward(net, eng):
        for q in range(3):
            gen = torch.Generator(device="cuda").manual_seed(q)
            x = torch.randn(16, 37, device="cuda", generator=gen).to(torch.bfloat16)
            eng.backward(net(x).float().square().sum(), q)

    net, eng = engine()
    with pytest.raises(RuntimeError):
        eng.clip_grad_norm(1.0)       # no gradients yet
    backward(net, eng)
    torch.cuda.synchronize()
    before = [s.double().clone() for s in eng.grad_shards]
    ref = math.sqrt(sum(float(s.pow(2).sum()) for s in before))
    assert ref > 1.0
    norm = eng.clip_grad_norm(0.5)
    torch.cuda.synchronize()
    assert abs(float(norm) - ref) <= 3e-6 * ref
    factor = 0.5 / (ref + 1e-6)
    for s, b in zip(eng.grad_shards, before):
        assert bool(((s.double() - b * factor).abs() <= 4e-6 * (b * factor).abs()).all())
    assert abs(float(eng.clip_grad_norm(0.5, "inf"))
               - max(float(b.abs().max()) if b.numel() else 0.0 for b in before) * factor) <= 1e-6
    eng.step()

    # a large limit changes nothing: the same bits as without the call
    net_a, eng_a = engine()
    net_b, eng_b = engine()
    backward(net_a, eng_a)
    backward(net_b, eng_b)
    eng_b.clip_grad_norm(1e9)
    eng_a.step()
    eng_b.step()
    torch.cuda.synchronize()
    assert torch.equal(eng_a.flat16, eng_b.flat16)


def test_engine_with_amp_refuses():
    net = torch.nn.Linear(8, 8).to("cuda", torch.float16)
    eng = ZeroEngine(net.parameters(), 2, amp=Z.AmpConfig())
    with pytest.raises(RuntimeError, match="max_norm"):
        eng.clip_grad_norm(1.0)
