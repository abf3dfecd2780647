"""Test helper: head norms with the rotation, token log probabilities and AdamW
through the library's binding, run once on the release library and once -- in a
child process -- on the access-checking build (librepops_debug.so), whose kernels
test every global access against the call's buffers.  The two must give the same
bytes, and the checked run must report no skipped access.

Usage as a child: python tests/checked_build_training_run.py <checked .so> <out .npz>
"""
import os
import sys

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

DEV = "cuda:0"


def workloads(rp):
    """Name -> host array of every result; raises if a kernel reported a skipped
    access or a timed-out wait."""
    import torch
    from verifiable_repops_gemm_gb300 import inputs
    out = {}
    kinds = (torch.float32, torch.float16, torch.bfloat16)

    def done(name, *ts):
        torch.cuda.synchronize()
        st = rp.device_status()
        if st != 0:
            raise RuntimeError("%s: device status %d" % (name, st))
        for i, t in enumerate(ts):
            if t is not None:
                out["%s.%d" % (name, i)] = t.detach().cpu().contiguous().view(-1).view(torch.uint8).numpy().copy()

    def rows(r, c, seed, pad=0, off=0, dt=torch.float32):
        # every tensor ends where its memory ends: what is read behind it is not its own
        flat = inputs.normal((max((r - 1) * (c + pad) + c, 1) + off,), 1.0, seed, DEV).to(dt)
        return flat.as_strided((r, c), (c + pad, 1), off)

    seed = 0
    for r, c in ((1, 1), (3, 33), (2, 255), (5, 1024), (3, 1025), (4, 5003), (1, 40001), (400, 2050)):
        for dt in kinds:
            for pad, off in ((0, 0), (1, 1), (8, 0), (3, 5)):
                seed += 1
                x = rows(r, c, seed, pad, off, dt)
                t = torch.arange(r, device=DEV) % c
                t[0] = -1
                a = rp.token_logprobs(x, t, temperature=0.8, top=min(c, 9))
                done("lp_%d" % seed, *a)
                w = inputs.normal((r,), 1.0, 5000 + seed, DEV)
                o = torch.zeros((r - 1) * (c + pad) + c + off, dtype=dt, device=DEV)
                o = o.as_strided((r, c), (c + pad, 1), off)
                done("lpb_%d" % seed, rp.token_logprobs_backward(x, t, a.stats, w, w, out=o),
                     rp.token_logprobs_backward(x, t, a.stats, w))
    for r, q, k, dim, pairs in ((1, 1, 1, 1, 0), (7, 3, 2, 80, 16), (40, 4, 1, 64, 32), (33, 2, 2, 7, 3), (9, 5, 1, 512, 256),
                                (3000, 16, 1, 4, 2)):
        for dt in kinds:
            for pad, off in ((0, 0), (3, 1), (4, 0)):
                for layout in ("adjacent", "halves"):
                    seed += 1
                    n = (q + k) * dim
                    x, dy = rows(r, n, 7000 + seed, pad, off, dt), rows(r, n, 8000 + seed, pad, off, dt)
                    cos, sin = (rows(50, pairs, 9000 + i, 0, 0) for i in (0, 1)) if pairs else (None, None)
                    g = dict(q_gain=inputs.normal((dim,), 1.0, 1, DEV), k_gain=inputs.normal((dim,), 1.0, 2, DEV))
                    pos = torch.arange(r, device=DEV) % 53 - 1          # one before the table, two behind it
                    o = torch.zeros((r - 1) * (n + pad) + n + off, dtype=dt, device=DEV).as_strided((r, n), (n + pad, 1), off)
                    kw = dict(layout=layout, positions=pos)
                    done("hn_%d" % seed, rp.head_norm_rope(x, q, k, cos, sin, out=o, **g, **kw).nan_to_num(3.0),
                         rp.head_norm_rope(x, q, k, cos, sin, inverse=True, **kw).nan_to_num(3.0))
                    done("hnb_%d" % seed, *(t.nan_to_num(3.0) for t in
                                            rp.head_norm_rope_backward(dy, x, q, k, cos, sin, dx=o, **g, **kw)))
    for bits in (32, 8):
        for dt in kinds:
            for k in (1, 3):
                for off in (0, 1):
                    seed += 1
                    sizes = [1, 127, 128, 129, 0, 4096, 9000] + [5] * 500
                    flat = lambda n, s, d=torch.float32: rows(1, max(n, 1), s, 0, off, d)[0][:n]
                    theta = [flat(n, 100 + i) for i, n in enumerate(sizes)]
                    grads = [[flat(n, 200 + i + 1000 * c, dt) for i, n in enumerate(sizes)] for c in range(k)]
                    st = rp.adamw_state(theta, bits)
                    for step in (1, 2):
                        rp.adamw(theta, grads, **st, step=step, lr=1e-2, weight_decay=0.1)
                    done("adam_%d" % seed, *theta[:8], *[t for ts in st.values() for t in ts[:8]])
                    if bits == 8:
                        done("adamm_%d" % seed, *rp.adamw_moments(*(ts[6] for ts in st.values())))
    return out


if __name__ == "__main__":
    import verifiable_repops_gemm_gb300 as rp
    from verifiable_repops_gemm_gb300 import _capi
    _capi.load(sys.argv[1])
    assert "-DREPOPS_DEBUG_BOUNDS" in rp.version(), rp.version()
    res = workloads(rp)
    np.savez(sys.argv[2], **res)
    print("checked run ok:", len(res), "results")
