"""The serving example against the same model run without pages: dense
attention over all tokens in 32 bits, everything recomputed for every step."""
import importlib.util
import os

import pytest
import torch

import paged_kv_decode_rope_gb300 as pkv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("serve_requests", os.path.join(ROOT, "examples", "serve_requests.py"))
    module = importlib.util.module_from_spec(spec)
    import sys
    sys.modules["serve_requests"] = module
    spec.loader.exec_module(module)
    return module


def dense_logits(ex, model, tokens):
    """The last token's logits after `tokens`, from scratch."""
    cfg = model.cfg
    n = len(tokens)
    pos = torch.arange(n, device="cuda")
    turn = pos[:, None].double() * torch.tensor(model.freqs, dtype=torch.float64, device="cuda")
    cos, sin = turn.cos()[:, None], turn.sin()[:, None]

    def rotate(x):
        y = x.double().clone()
        a, b = x[..., 0:cfg.rot_dim:2].double(), x[..., 1:cfg.rot_dim:2].double()
        y[..., 0:cfg.rot_dim:2] = (a * cos - b * sin) * model.magnitude
        y[..., 1:cfg.rot_dim:2] = (b * cos + a * sin) * model.magnitude
        return y.float()

    x = model.embed[torch.tensor(tokens, device="cuda")]
    for layer in range(cfg.layers):
        q, k, v = model.project(layer, x)
        q, k, v = rotate(q), rotate(k).to(torch.bfloat16).float(), v.float()
        group = cfg.q_heads // cfg.kv_heads
        k, v = k.repeat_interleave(group, 1), v.repeat_interleave(group, 1)
        s = torch.einsum("ihd,jhd->hij", q, k) * pkv.HEAD_DIM ** -0.5
        s = cfg.softcap * torch.tanh(s / cfg.softcap)
        seen = pos[None, :] <= pos[:, None]
        if layer % 2:
            seen &= pos[None, :] > pos[:, None] - cfg.window
        p = torch.softmax(s.masked_fill(~seen, float("-inf")), dim=-1)
        o = torch.einsum("hij,jhd->ihd", p, v).to(torch.bfloat16)
        x = x + o.reshape(n, -1) @ model.out[layer].T
    return model.logits(x[-1:])[0].float()


@pytest.mark.gpu
def test_the_example_agrees_with_the_dense_model():
    ex = example()
    cfg = ex.Config(layers=3, vocab=1009)
    model = ex.Model(cfg, seed=3)
    g = torch.Generator().manual_seed(4)
    prompts = [torch.randint(0, cfg.vocab, (n,), generator=g).tolist() for n in (3, 90, 17, 64, 1)]
    tokens, outs = ex.generate(model, prompts, 20)
    for b, prompt in enumerate(prompts):
        seen = list(prompt)
        for step, out in enumerate(outs):
            want = dense_logits(ex, model, seen)
            # bf16 activations on both sides, rounded in other places: a few roundings of 2^-8 of logits that
            # are sums of `width` products of unit-variance numbers
            got = out["logits"][b].float()
            assert (got - want).norm() <= 0.02 * want.norm(), (b, step)
            logp = torch.log_softmax(got.double(), dim=-1)
            assert torch.equal(out["top_ids"][b].long(), torch.sort(got, descending=True, stable=True).indices[:cfg.top])
            assert (out["top_logprobs"][b].double() - logp[out["top_ids"][b].long()]).abs().max() < 1e-4
            assert abs(float(out["entropy"][b]) - float(-(logp.exp() * logp).sum())) < 1e-4
            seen.append(int(tokens[step, b]))


@pytest.mark.gpu
def test_a_step_replays_from_a_graph():
    """The five calls of a decode step, captured once and replayed: the same as run one by one."""
    ex = example()
    cfg = ex.Config(layers=2, vocab=701)
    model = ex.Model(cfg, seed=5)
    i32 = dict(dtype=torch.int32, device="cuda")

    def server():
        torch.manual_seed(6)
        s = ex.Server(model, 3, 64, 60)
        s.step(torch.arange(60, **i32), torch.tensor([20, 39, 1], **i32), one_each=False)
        return s

    tokens, one = torch.tensor([5, 6, 7], **i32), torch.ones(3, **i32)
    a = server()
    want = a.step(tokens, one, one_each=True)
    b = server()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # (library handles of the projections are made outside the capture)
        model.project(0, model.embed[:3])
        model.logits(model.embed[:3])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = b.step(tokens, one, one_each=True)
    for _ in range(2):  # the same step again: it appends the same tokens in the same slots
        graph.replay()
        torch.cuda.synchronize()
        for name in want:
            assert torch.equal(want[name], got[name]), name
    assert a.error_bits() == 0 and b.error_bits() == 0
    a.close()
    b.close()


def test_the_example_is_documented():
    text = open(os.path.join(ROOT, "README.md"), encoding="utf-8").read()
    assert "examples/serve_requests.py" in text
