"""The windowed decode's workspace is planned for the cache's device, as the call
itself plans, whichever device is current."""

import types

import numpy as np

import bit_mla_kv_lowbit_gb300 as pkg


def test_the_plan_is_that_of_the_caches_device(monkeypatch):
    import torch
    cache = pkg.PagedCache(4, 4, np.zeros((2, 512), np.int32), 4, device="cpu")
    plan, asked = pkg.window_plan, []

    def properties(device):
        asked.append(device)
        return types.SimpleNamespace(multi_processor_count=20)
    sizes = []
    monkeypatch.setattr(torch.cuda, "get_device_properties", properties)
    monkeypatch.setattr(pkg.binding, "decode_window", lambda lay, q, pool, table, lens, sink, recent, out, ws, *a, **k:
                        sizes.append(ws.numel()))
    q = torch.zeros(2, 16, 576, dtype=torch.bfloat16)
    for _ in range(2):
        cache.decode_window(q, torch.zeros(2, dtype=torch.int32), 0.1, 1 << 20, sinks=3)
    want = plan(cache.layout, 2, 16, 1, 1 << 20, 3, 512, num_sms=20)[1]
    assert want != plan(cache.layout, 2, 16, 1, 1 << 20, 3, 512, num_sms=152)[1]
    assert sizes == [want, want]
    assert asked == [cache.pool.device]  # once a cache
