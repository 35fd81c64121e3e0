"""The voxel-transformer block of examples/voxel_block.py: forward and every
gradient against the same block in 64 bits with autograd, and its training
step replayed from a captured graph.

Tolerances.  The longest chain from input to gradient rounds about 20 times
to the feature type; a rounding moves a tensor by at most u of its norm (u =
2^-11 fp16, 2^-8 / 2 bf16), and the maps in between neither shrink nor raise
relative errors: 20 u.  What goes through 8 bits (x for the first norm's
backward pass, the convolution's input for its weight gradient) is a multiple
of a quantum q with the block's largest value at least 64 q; the error's rms
is q / sqrt(12), and the rms of 32 normal values is over a third of their
largest one: 0.29 / (64 / 3) = 0.014 of the norm more."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import bench
import oracle
from convolution_voxelised_point_amd import synth

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
UNIT = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -9}
EIGHT = 0.014


@pytest.fixture(scope="module")
def vb(ts):
    spec = importlib.util.spec_from_file_location("voxel_block", os.path.join(ROOT, "examples", "voxel_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def exact(block, coords, starts, p, x):
    """The block in 64 bits, on the CPU."""
    def norm(h, w):
        return h * torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-6) * w
    n, c = x.shape
    hq, hk, d = block.hq, block.hk, block.d
    q, k, v = (norm(x, p.norm1) @ p.qkv).view(n, hq + 2 * hk, d).split((hq, hk, hk), dim=1)
    k, v = (t.repeat_interleave(hq // hk, dim=1) for t in (k, v))
    att = []
    for a, b in zip(starts[:-1], starts[1:]):
        pos = coords[a:b, 1:].double()
        dist = (pos[:, None] - pos[None]).square().sum(-1).sqrt()
        for h in range(hq):
            z = q[a:b, h] @ k[a:b, h].T * d ** -0.5 - block.slopes[h].item() * dist
            att.append(torch.softmax(z, 1) @ v[a:b, h])
    rows = [torch.cat(att[i:i + hq], 1) for i in range(0, len(att), hq)]
    h = x + torch.cat(rows) @ p.out
    n2 = norm(h, p.norm2)
    t_in, t_out, t_off = (torch.from_numpy(np.asarray(t)).long() for t in oracle.kmap(coords.numpy(), coords.numpy(), 3, 1))
    y = h
    for o in range(27):
        at = t_off == o
        y = y.index_add(0, t_out[at], n2[t_in[at]] @ p.conv[o])
    return y


CASES = [("f16", torch.float16, 32, 4, 2), ("bf16", torch.bfloat16, 64, 4, 1), ("odd_heads", torch.float16, 60, 5, 5)]


@pytest.mark.parametrize("name,dtype,c,hq,hk", CASES, ids=[c[0] for c in CASES])
def test_block_against_64_bits(vb, name, dtype, c, hq, hk):
    coords = synth.random_coords(40, 500, 3, 2, 9)
    scene, block = vb.Scene.of(coords, 4), vb.Block(c, hq, hk)
    low = vb.typed(block.init(5), dtype)
    g = torch.Generator("cuda").manual_seed(6)
    x, dy = (torch.randn(len(coords), c, generator=g, device="cuda").to(dtype) for _ in range(2))
    y, saved = block.forward(scene, low, x)
    dx, grads = block.backward(scene, low, saved, dy)

    ref = vb.Params(*(t.double().cpu().requires_grad_() for t in low))
    xr = x.double().cpu().requires_grad_()
    yr = exact(block, scene.coords.cpu(), scene.starts.tolist(), ref, xr)
    yr.backward(dy.double().cpu())

    tol = 20 * UNIT[dtype]
    checks = [("y", y, yr, tol), ("dx", dx, xr.grad, tol + EIGHT)]
    for field in vb.Params._fields:
        bar = tol + (EIGHT if field in ("norm1", "conv") else 0.0)
        checks.append((field, getattr(grads, field), getattr(ref, field).grad, bar))
    for what, got, want, bar in checks:
        want = want.detach()
        err = float((got.double().cpu() - want).norm() / want.norm())
        assert err <= bar, f"{what}: {err} > {bar}"


def test_step_replays_from_a_graph(vb, ts):
    coords = synth.random_coords(41, 3000, 3, 1, 20)
    scene, block = vb.Scene.of(coords, 8), vb.Block(64, 4, 2)
    low = vb.typed(block.init(7), torch.bfloat16)
    g = torch.Generator("cuda").manual_seed(8)
    x, dy = (torch.randn(len(coords), 64, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    held = []

    def step():
        y, saved = block.forward(scene, low, x)
        held[:] = [y, block.backward(scene, low, saved, dy)]
    step()
    flat = lambda: [held[0], held[1][0], *held[1][1]]
    want = [t.clone() for t in flat()]
    graph = bench.capture([step])
    for _ in range(3):
        a = torch.randn(512, 512, device="cuda")
        (a @ a).sum().item()  # unrelated eager work and a synchronisation
        for t in flat():
            t.fill_(-7)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for got, t in zip(flat(), want):
            assert torch.equal(got, t)


@pytest.mark.parametrize("d,first", [(16, 0), (12, 0), (16, 4)])
def test_gradients_into_columns(vb, ts, d, first):
    """Gradients written to the columns of one matrix are those written apart, also where the columns do not
    begin at 16 bytes; other layouts are refused."""
    n, hq, hk = 70, 4, 2
    g = torch.Generator("cuda").manual_seed(9)
    wide = (hq + 2 * hk) * d
    m = torch.randn(n * wide + first, generator=g, device="cuda").half()[first:].view(n, wide)
    heads = lambda t: t.view(n, -1, d).split((hq, hk, hk), dim=1)
    starts = torch.tensor([0, 33, 33, 70], device="cuda")
    out, lse = ts.attn_fwd(*heads(m), starts)
    dout = torch.randn(n, hq, d, generator=g, device="cuda").half()
    apart = ts.attn_bwd(dout, *heads(m), out, lse, starts)
    dm = torch.full((n * wide + first,), float("nan"), device="cuda", dtype=m.dtype)[first:].view(n, wide)
    got = ts.attn_bwd(dout, *heads(m), out, lse, starts, into=heads(dm))
    assert torch.equal(dm.view(n, -1, d), torch.cat(apart, 1))
    assert [t.data_ptr() for t in got] == [t.data_ptr() for t in heads(dm)]
    for wrong in ([t.contiguous() for t in heads(dm)], list(heads(dm.float())), list(heads(dm))[:2]):
        with pytest.raises(ts.TsError):
            ts.attn_bwd(dout, *heads(m), out, lse, starts, into=wrong)
