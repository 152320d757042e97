"""The block norms where fp32 ends: an eps below its normal numbers with rows of zeros, whose root is then
taken of eps alone, and rows whose sum of squares is near the largest number."""
import numpy as np
import pytest
import torch

import gated_delta_rule_78_amd as kda
from oracle import block_norm
from tests.parity import host32, say
from tests.test_gpu_block_norm import BF16, F32, check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("eps,pre_eps", [(1e-40, 1e-5), (1e-6, 3e-44), (1.4e-45, 1e-6)])
@pytest.mark.parametrize("D,dt", [(24, F32), (128, BF16), (1000, F32), (1001, BF16), (4096, BF16), (12000, F32)])
def test_subnormal_eps(D, dt, eps, pre_eps):
    """Each output against the formula: 1 / sqrt(eps) is up to 2.7e22 and finite, and times zero is zero."""
    say("eps %g %g, %d channels" % (eps, pre_eps, D))
    c = make(7, D, dt, dt, seed=11)
    c["f"][0] = 0
    c["x"][0] = 0
    c["f"][2] = 0
    c["f"][4] *= 2.0 ** -40                            # its mean square, 2^-80, is far above eps
    kw = dict(gate=c["gate"], norm_weight=c["w_post"], eps=eps, scale=0.7, scale_weight=c["lam"], pre_weight=c["w_pre"],
              pre_eps=pre_eps)
    got = dict(zip(("x_out", "n"), kda.block_norm_fwd(c["f"], c["x"], **kw)))
    got.update(zip(("df", "dx", "dgate", "dw_post", "dlam", "dw_pre"),
                   kda.block_norm_bwd(c["f"], c["x"], c["dxo"], c["dn"], **kw)))
    r32 = lambda v: float(np.float32(v))
    ref = block_norm.evaluate(*[host32(c[k]) for k in ("f", "x", "gate", "w_post", "lam", "w_pre")], post=True, pre=True,
                              scale=r32(0.7), eps=r32(eps), pre_eps=r32(pre_eps), dxo=host32(c["dxo"]), dn=host32(c["dn"]))
    for key, t in got.items():
        check("ends", t, ref, key, F32 if key in ("dw_post", "dlam", "dw_pre") else dt)
    assert not bool(got["x_out"][0].any()) and not bool(got["n"][0].any())


@pytest.mark.parametrize("D,dt", [(64, F32), (1001, BF16), (4096, BF16), (16384, F32)])
def test_largest_values(D, dt):
    """Rows whose sum of squares is just finite: 3/4 of the largest number in fp32, in f and in x_out."""
    say("largest values, %d channels" % D)
    c = make(3, D, dt, F32, gate=False, seed=12)
    big = (0.75 * 2.0 ** 128 / D) ** 0.5
    c["f"][0] = (torch.where(c["f"][0] < 0, -big, big) * (1 - 2.0 ** -8)).to(dt)      # rounds to at most big
    c["x"][1] = torch.where(c["x"][1] < 0, -big, big)
    kw = dict(norm_weight=c["w_post"], eps=1e-6, scale=0.7, scale_weight=c["lam"], pre_weight=c["w_pre"], pre_eps=1e-6)
    got = dict(zip(("x_out", "n"), kda.block_norm_fwd(c["f"], c["x"], **kw)))
    got.update(zip(("df", "dx"), kda.block_norm_bwd(c["f"], c["x"], c["dxo"], c["dn"], **kw)[:2]))
    r32 = lambda v: float(np.float32(v))
    ref = block_norm.evaluate(*[host32(c[k]) if c[k] is not None else None for k in ("f", "x", "gate", "w_post", "lam", "w_pre")],
                              post=True, pre=True, scale=r32(0.7), eps=r32(1e-6), pre_eps=r32(1e-6), dxo=host32(c["dxo"]),
                              dn=host32(c["dn"]))
    for key, t in got.items():
        check("ends", t, ref, key, dt if key in ("n", "df") else F32)
