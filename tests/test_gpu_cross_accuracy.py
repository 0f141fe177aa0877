"""The norm of cross attention's bf16 errors in every form of the kernels: what independent
roundings of P, dS and the results add up to (rounding_norms.py), and not more."""
import pytest
import torch

import block_reference as ref
from parity import record_margin
from rounding_norms import error_norms, limits
from test_gpu_cross import FORMS, run, tokens

pytestmark = pytest.mark.gpu

# single tokens and split states; the many-row forms of each head size; groups
SIZES = FORMS + [(4, 1, 5000, 8, 2, 64), (1, 16, 5000, 1, 1, 32), (2, 1030, 2900, 6, 2, 32), (1, 131, 33000, 4, 4, 32),
                 (2, 1100, 4097, 2, 1, 64), (2, 450, 2300, 6, 2, 128), (40, 784, 196, 4, 4, 32), (1, 2000, 513, 5, 5, 128)]


@pytest.mark.parametrize("means", [(0.0, 0.0), (0.5, 1.0)], ids=["centred", "offset"])
@pytest.mark.parametrize("masked", [False, True], ids=["all", "mask"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_errors_are_the_roundings(size, masked, means):
    B, Lq, Lk, h, kv, d = size
    t = torch.bfloat16
    q, g = tokens(1, B, Lq, h * d, dtype=t), tokens(4, B, Lq, h * d, dtype=t)
    k, v = tokens(2, B, Lk, kv * d, dtype=t, mean=means[0]), tokens(3, B, Lk, kv * d, dtype=t, mean=means[1])
    m = None
    if masked:
        m = (torch.rand((B, Lk), generator=torch.Generator(device="cuda").manual_seed(5), device="cuda") < 0.6)
    ok = ref.valid_states(B, Lk, None, m, "cuda")
    r = ref.cross(q, k, v, h, kv, ok, None, g)
    most = limits(error_norms(q, k, v, h, kv, ok, r, g), r)
    out = run(q, k, v, h, kv, None, m, g)
    for x, limit in most.items():
        share = float((out[x].double() - r[x]).norm()) / limit
        record_margin(f"norm {size} {x}", share, 1.0)
        assert share <= 1.0, f"{x}: {share:.3f} of the roundings' norm"
