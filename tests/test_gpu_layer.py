"""The layer with experts of examples/voxel_block.py, which runs the rotation, attention, the
router, the grouped products and the combining sum together: forward and every gradient against
the same layer in 64 bits with autograd, and its training step replayed from a captured graph.

Tolerances as those of the block's test: the longest chain rounds about 24 times to the feature
type, each time by at most u of the tensor's norm (u = 2^-11 fp16, 2^-9 bf16), the maps between
neither shrink nor raise relative errors: 24 u; what goes through 8 bits (x for the first norm's
backward pass) adds 0.014.  Which experts a voxel takes is a matter of the logits as they
are: the reference is told."""
import importlib.util
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import bench
from convolution_voxelised_point_amd import synth

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
UNIT = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -9}


@pytest.fixture(scope="module")
def vb(ts):
    spec = importlib.util.spec_from_file_location("voxel_block_layer", os.path.join(ROOT, "examples", "voxel_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def exact(layer, coords, starts, p, x, experts):
    """The layer in 64 bits, on the CPU, with the given experts of each voxel."""
    def norm(h, w):
        return h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6) * w
    n, c = x.shape
    hq, hk, d = layer.hq, layer.hk, layer.d
    q, k, v = (norm(x, p.norm1) @ p.qkv).view(n, hq + 2 * hk, d).split((hq, hk, hk), dim=1)
    axis = np.repeat(np.arange(3), layer.pairs)
    angle = coords[:, 1:].double()[:, axis] * layer.freqs.cpu().double()
    cos, sin, half = torch.cos(angle)[:, None], torch.sin(angle)[:, None], d // 2

    def turn(t):
        a, b = t[..., :half], t[..., half:]
        return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    q, k = turn(norm(q, p.norm_q)), turn(norm(k, p.norm_k))
    k, v = (t.repeat_interleave(hq // hk, dim=1) for t in (k, v))
    rows = []
    for a, b in zip(starts[:-1], starts[1:]):
        z = torch.matmul(q[a:b].transpose(0, 1), k[a:b].permute(1, 2, 0)) * d ** -0.5
        rows.append(torch.matmul(torch.softmax(z, 2), v[a:b].transpose(0, 1)).transpose(0, 1).reshape(b - a, hq * d))
    h = x + torch.cat(rows) @ p.out
    n2 = norm(h, p.norm2)
    gates = torch.softmax((n2 @ p.router).gather(1, experts), 1)
    y = h
    for e in range(layer.experts):
        t, j = torch.nonzero(experts == e, as_tuple=True)
        a, b = (n2[t] @ p.up[e]).chunk(2, 1)
        y = y.index_add(0, t, gates[t, j][:, None] * ((torch.nn.functional.silu(a) * b) @ p.down[e]))
    return y


# channels, heads, key-value heads, experts, hidden, top
CASES = [("f16", torch.float16, 32, 4, 2, 4, 48, 2), ("bf16", torch.bfloat16, 64, 4, 1, 16, 128, 3), ("odd", torch.float16, 60, 5, 5, 3, 37, 1),
         ("idle", torch.bfloat16, 64, 2, 2, 40, 64, 2)]


@pytest.mark.parametrize("name,dtype,c,hq,hk,experts,hidden,top", CASES, ids=[c[0] for c in CASES])
def test_layer_against_64_bits(vb, name, dtype, c, hq, hk, experts, hidden, top):
    coords = synth.random_coords(50, 500, 3, 2, 9)
    scene, layer = vb.Scene.of(coords, 4), vb.Layer(c, hq, hk, experts, hidden, top)
    p = layer.init(15)
    if name == "idle":  # most experts get nothing
        p.router[:, 5:] = 0.0
        p.router[:, :5] *= 4.0
    low = vb.typed(p, dtype)
    g = torch.Generator("cuda").manual_seed(16)
    x, dy = (torch.randn(len(coords), c, generator=g, device="cuda").to(dtype) for _ in range(2))
    y, saved = layer.forward(scene, low, x)
    counts = saved.route.starts.diff()
    assert int(counts.sum()) == len(coords) * top
    dx, grads = layer.backward(scene, low, saved, dy)

    ref = vb.LayerParams(*(t.double().cpu().requires_grad_() for t in low))
    xr = x.double().cpu().requires_grad_()
    yr = exact(layer, scene.coords.cpu(), scene.starts.tolist(), ref, xr, saved.route.experts.cpu().long())
    yr.backward(dy.double().cpu())
    tol = 24 * UNIT[dtype]
    checks = [("y", y, yr, tol), ("dx", dx, xr.grad, tol + 0.014)]
    for field in vb.LayerParams._fields:
        checks.append((field, getattr(grads, field), getattr(ref, field).grad, tol + (0.014 if field == "norm1" else 0.0)))
    for what, got, want, bar in checks:
        want = want.detach()
        if float(want.norm()) == 0.0:
            assert float(got.double().norm()) == 0.0, what  # one expert a voxel: its gate is 1
            continue
        err = float((got.double().cpu() - want).norm() / want.norm())
        assert err <= bar, f"{what}: {err} > {bar}"


def test_step_replays_from_a_graph(vb, ts):
    coords = synth.random_coords(51, 3000, 3, 1, 20)
    scene, layer = vb.Scene.of(coords, 8), vb.Layer(64, 4, 2, 8, 128)
    low = vb.typed(layer.init(17), torch.bfloat16)
    g = torch.Generator("cuda").manual_seed(18)
    x, dy = (torch.randn(len(coords), 64, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    held = []

    def step():
        y, saved = layer.forward(scene, low, x)
        held[:] = [y, layer.backward(scene, low, saved, dy)]
    step()
    flat = lambda: [held[0], held[1][0], *held[1][1]]  # noqa: E731
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


def test_two_graphs_share_nothing(ts):
    """A pass through the library's operators, captured twice with other inputs and replayed on two streams at
    once.  (Without torch's matrix products, whose workspace belongs to the stream they were captured on.)"""
    def made(seed, n, e, c):
        g = torch.Generator("cuda").manual_seed(seed)
        normal = lambda *s, dt=torch.bfloat16: torch.randn(*s, generator=g, device="cuda").to(dt)  # noqa: E731
        q, k, dq, dk, dy, logits = normal(n, 4, 32), normal(n, 2, 32), normal(n, 4, 32), normal(n, 2, 32), normal(n, c), normal(n, e)
        w = normal(32, dt=torch.float32)
        coords = torch.randint(0, 500, (n, 4), generator=g, device="cuda", dtype=torch.int32)
        freqs, pairs = ts.rope_freqs((6, 6, 4)), (6, 6, 4)
        x, up, down = normal(n, c), normal(e, c, 4 * c), normal(e, 2 * c, c)
        held = []

        def step():
            r = ts.route_fwd(logits, 2)
            own, groups = ts.Groups(r.starts), ts.Groups(r.starts, r.rows)
            t, h = ts.group_glu_fwd(x, up, groups, want_h=True)
            z = ts.group_fwd(t, down, own)
            dz, dg = ts.combine_bwd(dy, z, r.place, r.gates)
            dh = ts.group_glu_dgrad(dz, down, h, own)
            held[:] = [*r, ts.combine_fwd(z, r.place, r.gates), dg, ts.route_bwd(dg, logits, r), ts.group_wgrad(t, dz, own),
                       ts.group_wgrad(x, dh, groups), ts.combine_fwd(ts.group_dgrad(dh, up, groups), r.place),
                       *ts.rope_fwd(q, k, coords, freqs, pairs, wq=w, wk=w), *ts.rope_bwd(dq, dk, q, k, coords, freqs, pairs, wq=w, wk=w)]
        step()
        want = [t.clone() for t in held]
        return bench.capture([step]), held, want, (q, k, dq, dk, dy, logits, w, coords, freqs, x, up, down)
    steps = [made(61, 9000, 6, 64), made(62, 5000, 9, 96)]
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(4):
        for _, held, _, _ in steps:
            for t in held:
                t.fill_(-7)
        torch.cuda.synchronize()
        for (graph, *_), stream in zip(steps, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for _, held, want, _ in steps:
            assert all(torch.equal(a, b) for a, b in zip(held, want))


def test_example_runs(ts):
    """The training command, with and without experts."""
    for extra in ([], ["--experts", "6"]):
        r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "voxel_block.py"), "--steps", "2", "--scale", "0.02", *extra],
                           capture_output=True, text=True, timeout=100)
        assert r.returncode == 0, r.stderr[-2000:]
        assert r.stdout.count("loss") == 2
