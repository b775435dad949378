"""GPU parity: the router's backward where the number of experts is no multiple
of the wave's 64 lanes and a token takes more experts than the last lanes hold,
vs the fp64 oracle (oracle/router.py)."""

import numpy as np
import pytest
import torch

import mxfp8_block_scaled_07_amd as mxa
import workloads
from oracle import router, routing

from gpu_util import dev, host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E,k", [(68, 8), (100, 64), (65, 2), (5, 5), (130, 3)])
def test_every_pair_reaches_its_expert(E, k):
    T, H = 40, 96
    g = np.random.default_rng([E, k])
    oi, ow = router.route_topk(g.standard_normal((T, E)).astype(np.float32), k)
    w = ow.astype(np.float32)
    _, _, dst, src = routing.route(oi, E, workloads.capacity(T, k, E))
    y = workloads.normal_bf16(g, (src.size, H), 1.0)
    d = workloads.normal_bf16(g, (T, H), 1.0)
    _, dl = mxa.router_bwd(dev(d), dev(y), dev(dst), dev(oi), dev(w), E)
    torch.cuda.synchronize()
    _, _, want, S = router.router_bwd(d, y, dst, oi, w, E)
    # each lane adds 8 products of H / 512 chunks, the wave 64 sums in 6 steps, the softmax's sum k in 6 more
    off = np.abs(host(dl) - want) > (H / 64 + 24) * 2.0 ** -24 * S + 2.0 ** -126
    assert not off.any(), np.argwhere(off)[:5]
