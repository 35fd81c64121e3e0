"""Resource records of the kernels beside the convolutions, as
test_kernel_resources.py reads them."""
import os
import re

from convolution_voxelised_point_amd import build as B
from test_kernel_resources import records


def test_every_source_with_kernels_reports_them():
    recs = records()
    for src in B.sources():
        with open(src) as f:
            kernels = set(re.findall(r"__global__[^;{]*?\b(k_\w+)\s*\(", f.read()))
        name = os.path.basename(src)
        for k in kernels:
            assert any(k in n for n in recs[name]), f"{name}: no record of {k}"
        for n, r in recs[name].items():
            for field in ("vgprs", "scratch_bytes", "lds_bytes", "waves_per_simd"):
                assert field in r, f"{name} {n}: {field} missing"
    assert {"act8.hip", "attn_bwd.hip", "attn_fwd.hip", "norm.hip", "wgrad.hip"} <= {s for s, r in recs.items() if r}


def test_attention_kernels_keep_their_waves():
    """The occupancy that launch.h plans for the windows' kernels (32 channels, biased)."""
    recs = {**records()["attn_fwd.hip"], **records()["attn_bwd.hip"]}
    for kernel, waves in (("k_attn_fwdI.*Li32ELi1ELb0ELb1ELb0ELb0E", 5), ("k_attn_dqI.*Li32ELi1ELb0ELb1ELb0ELb1E", 3),
                          ("k_attn_dkvI.*Li32ELi1ELb0ELb1E", 3)):
        found = [n for n in recs if re.search(kernel, n)]
        assert len(found) == 2, (kernel, found)  # fp16 and bf16
        for n in found:
            assert recs[n]["waves_per_simd"] >= waves, (n, recs[n])
