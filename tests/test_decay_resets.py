"""Log-decays that reset the state (large magnitudes, the type's lowest value, -infinity) on every path of the
chunked rule, forward and backward: the tokens behind a reset decay among themselves as ever.

Tolerances: those of test_bwd_rule.py, and the method's for the forward (gdn_testutil.py).  Three tokens count as
-256 here, two of them in one chunk: their cumulative sum of about 530 has an fp32 spacing of 6e-5, so a
decay between later tokens of that chunk is off by at most 3e-5 of itself, under the 1e-4 of the fp32 forward."""
import pytest
import torch

import bwd_reference as ref
from gdn_testutil import BF16_REL_L2, F32_REL, rel_l2
from test_bwd_rule import F32_TOL, TC_TOL, call, make
from gated_deltanet_fwd_b200 import gdn

pytestmark = pytest.mark.gpu
RESETS = [-300.0, -1e4, -1e6, -1e9, -3.4028234663852886e38, float("-inf")]
PATHS = [("bf16", 128, 64), ("bf16", 128, 32), ("bf16", 48, 16), ("f32", 64, 32), ("f32", 128, 64)]


def resetting(dtype, d, value, T=300):
    x = make([T], 1, 2, d, d, dtype, True, a_mean=-6.0, seed=7)
    x["g"][[40, 41, 130]] = value
    return x


@pytest.mark.parametrize("value", RESETS)
@pytest.mark.parametrize("dtype,d,chunk", PATHS)
def test_gradients(dtype, d, chunk, value):
    x = resetting(dtype, d, value)
    got = call(x, chunk)
    want = ref.rule_grads(x, [300], d ** -0.5)
    tol = F32_TOL if dtype == "f32" else TC_TOL if (d, chunk) == (128, 64) else 2.0 ** -8 + F32_TOL
    for n, y in zip(("dq", "dk", "dv", "dg", "dbeta", "dS0"), got):
        r = rel_l2(y.reshape(want[n].shape), want[n])
        assert r <= tol, (n, r)
    dg = ref.d64(got[3]).reshape(300, 2)
    assert (dg[[40, 41, 130]].abs() <= tol * dg.abs().max()).all()


@pytest.mark.parametrize("value", RESETS)
@pytest.mark.parametrize("dtype,d,chunk,small_workspace", [(*p, False) for p in PATHS] + [("bf16", 128, 64, True)])
def test_forward(dtype, d, chunk, small_workspace, value):
    x = resetting(dtype, d, value)
    c = lambda n: x[n][None].cuda()
    ws = torch.empty(256, dtype=torch.uint8, device="cuda") if small_workspace else None
    out, S = gdn.gdn_chunk_fwd(c("q"), c("k"), c("v"), c("g"), c("beta"), initial_state=x["S0"].cuda(), chunk=chunk,
                               workspace=ws)
    want, Sw = ref.rule(*(ref.d64(x[n]) for n in ("q", "k", "v", "g", "beta")), d ** -0.5, ref.d64(x["S0"]), [300])
    tol = BF16_REL_L2 if dtype == "bf16" else F32_REL
    assert rel_l2(out[0], want) <= tol and rel_l2(S, Sw) <= tol


@pytest.mark.parametrize("value", [-1e9, float("-inf")])
def test_long_sequence(value):
    """Long enough for the forward's segments to be composed."""
    x = resetting("bf16", 128, value, T=3000)
    x["g"][1500] = x["g"][2990] = value
    c = lambda n: x[n][None].cuda()
    out, S = gdn.gdn_chunk_fwd(c("q"), c("k"), c("v"), c("g"), c("beta"), initial_state=x["S0"].cuda())
    want, Sw = ref.rule(*(ref.d64(x[n]) for n in ("q", "k", "v", "g", "beta")), 128 ** -0.5, ref.d64(x["S0"]), [3000])
    assert rel_l2(out[0], want) <= BF16_REL_L2 and rel_l2(S, Sw) <= BF16_REL_L2


@pytest.mark.parametrize("dtype,d,chunk", PATHS)
def test_nan_stays_nan(dtype, d, chunk):
    x = resetting(dtype, d, float("nan"))
    c = lambda n: x[n][None].cuda()
    out, S = gdn.gdn_chunk_fwd(c("q"), c("k"), c("v"), c("g"), c("beta"), initial_state=x["S0"].cuda(), chunk=chunk)
    assert out[0, 40:].isnan().any(-1).all() and S.isnan().all()
    assert call(x, chunk)[5].isnan().all()
