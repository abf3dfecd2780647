"""AdamW over lists in which tensors without elements fill a whole launch's table:
496 of them with one gradient, three with 1024 contributors."""
import pytest
import torch

import adamw_ref as ref
from test_gpu_adamw import DEV, HYPER, host, problem, restored, same

pytestmark = pytest.mark.gpu

LISTS = [([7] + [0] * 600 + [5], 1), ([0] * 1200 + [5], 1), ([7] + [0] * 1200, 1), ([0] * 495 + [9, 0, 130], 1),
         ([0] * 496 + [4097], 1), ([3] + [0] * 991 + [2, 0], 1), ([0, 0, 0, 0, 5], 1024), ([6, 0, 0, 0, 0], 1024),
         ([300, 0, 0, 0, 0, 0, 0, 1], 1024)]


@pytest.mark.parametrize("sizes,k", LISTS, ids=lambda v: str(len(v)) if isinstance(v, list) else str(v))
@pytest.mark.parametrize("bits", [32, 8])
def test_tables_of_empty_tensors(rp, sizes, k, bits):
    theta, grads, st = problem(sizes, 1, "f32", 5, bits=bits)
    moments = [restored(st, i) if bits == 8 else (host(st["m"][i]), host(st["v"][i])) for i in range(len(sizes))]
    was = [host(t) for t in theta]
    rp.adamw(theta, grads * k if k > 1 else grads[0], **st, step=3, lr=1e-2, weight_decay=0.1, seed=2, **HYPER)
    sc = ref.scalars(3, 1e-2, HYPER["betas"], 2)
    for i, n in enumerate(sizes):
        if n == 0:
            continue
        m, v = moments[i]
        want = ref.step(was[i], [host(grads[0][i])] * k, m, v * v if bits == 8 else v, sc, 0.1, HYPER["betas"], HYPER["eps"])
        assert same(host(theta[i]), want[0])
        if bits == 32:
            assert same(host(st["m"][i]), want[1]) and same(host(st["v"][i]), want[2])
        else:                                # the dither is keyed by the place among all of them
            dm, dr = ref.dither(n, sc[3], i)
            got = restored(st, i)
            assert same(got[0], ref.coded(want[1], False, dm)[0]) and same(got[1], ref.coded(want[3], True, dr)[0])
    assert torch.cuda.current_device() == torch.device(DEV).index
