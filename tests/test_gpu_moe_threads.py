"""The sort by expert from several host threads at once."""
import threading

import pytest
import torch

import activated_mlp_gemms_gb300 as m

pytestmark = pytest.mark.gpu


def test_threads_with_different_numbers_of_experts():
    # each thread's sort takes its own shared memory, whatever the others' launches take
    errors, start = [], threading.Barrier(4)

    def run(E):
        try:
            p = m.moe(64, E, 1, 8)
            ids = (torch.arange(64, device="cuda") * 7 % E).int().view(64, 1)
            plan = m.alloc_moe_plan(p)
            start.wait()
            for _ in range(3000):
                m.mlp_moe_sort(p, ids, plan)
            torch.cuda.synchronize()
            pos = m.moe_plan_views(p, plan)["pos"]
            assert (pos >= 0).all() and pos.unique().numel() == 64
        except Exception as e:  # noqa: BLE001 (shown below)
            errors.append((E, repr(e)))

    threads = [threading.Thread(target=run, args=(E,)) for E in (1024, 384, 700, 400)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
