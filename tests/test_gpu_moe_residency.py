"""GPU test of the routed layer on an expert cache: the residency as ft_expert_cache_where tells it, one device table a layer, and
the cache's slots as the records."""
import numpy as np
import pytest

from moe_expert_offload_amd import ft
from moe_expert_offload_amd.synth import Shape, Workload, allowed_mask, expert_record, generator, router_weights, tokens, zipf_reuse_trace
from tests import dense_ref as R
from tests import moe_ref as M
from tests.gpu_helpers import Engine, PinnedPool, dev, dev_u16, torch_mod

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,T", [("bf16", 2), ("mxfp4", 5), ("bf16", 40)])
def test_device_part_of_a_cached_layer(fmt, T):
    torch = torch_mod()
    print("[case] moe residency", fmt, T, flush=True)
    wl = Workload("residency", 33, Shape(3, 12, 256, 128, 3, fmt == "mxfp4"), 1, 0.5)
    s = wl.shape
    pool = PinnedPool(s, s.L * s.E)
    wr = [router_weights(wl, l) for l in range(s.L)]
    if fmt == "mxfp4":
        pool.fill_device_random(33)
    else:
        for r in range(s.L * s.E):
            pool.view[r] = expert_record(wl, r // s.E, r % s.E)
    eng = Engine(s, pool, 20, T_max=4, frac_q16=30000, max_fetch=2, cpu_threads=4)
    try:
        tr = zipf_reuse_trace(s.L, s.E, s.k, 1, 6, 1.1, 0.5, generator(33, 3))
        for step in range(6):
            for l in range(s.L):
                y = torch.empty((1, s.d), dtype=torch.float32, device="cuda")
                ft.ft_moe_decode_layer(eng.ctx, l, dev_u16(tokens(wl, step, l)), 1, dev_u16(wr[l]),
                                       dev(allowed_mask(tr[step, l], s.E)), y, plan=ft.ft_plan())
        torch.cuda.synchronize()
        shape = ft.make_shape(1, s.E, s.d, s.d_ff, s.k, ft.FT_W_MXFP4 if s.mxfp4 else ft.FT_W_BF16)
        wsb = ft.ft_moe_layer_workspace_bytes(shape, T)
        ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
        absent = 0
        for l in range(s.L):
            where = [ft.ft_expert_cache_where(eng.ctx, l, e) for e in range(s.E)]
            x = dev_u16(tokens(wl, 50, l, T=T))
            y = torch.empty((T, s.d), dtype=torch.float32, device="cuda")
            idx = torch.empty((T, s.k), dtype=torch.int32, device="cuda")
            gates = torch.empty((T, s.k), dtype=torch.float32, device="cuda")
            ft.ft_moe_layer(shape, x, T, dev_u16(wr[l]), None, eng.slots, 20, dev(np.array(where, np.int32)), None, y, ft.FT_T_FP32,
                            idx, gates, ws, wsb)
            torch.cuda.synchronize()
            recs = torch.from_numpy(pool.view[l * s.E:(l + 1) * s.E].copy().view(np.uint8).reshape(s.E, -1))
            here = {e: e for e in range(s.E) if where[e] >= 0}
            absent += sum(e not in here for e in idx.flatten().tolist())
            want = M.layer(x.cpu().view(torch.bfloat16), recs, here, idx.cpu(), gates.cpu(), s.d, s.d_ff, fmt, torch.float32)
            R.check(y, want, "y")
        assert absent > 0  # the tables left some of the taken experts out
    finally:
        eng.destroy()
        pool.free()
