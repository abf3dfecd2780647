"""Test helper: the 8-bit product, the 8-bit rows and the block edge through the
library's binding, run once on the release library and once -- in a child
process -- on the access-checking build (librepops_debug.so), whose kernels test
every global access against the call's buffers.  The two must give the same
bytes, and the checked run must report no skipped access.

Usage as a child: python tests/checked_build_rows8_run.py <checked .so> <out .npz>
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

    def done(name, *ts):
        torch.cuda.synchronize()
        st = rp.device_status()
        if st != 0:
            raise RuntimeError("%s: device status %d" % (name, st))
        for i, t in enumerate(ts):
            if t is not None:
                out["%s.%d" % (name, i)] = t.detach().cpu().contiguous().view(torch.uint8).numpy().copy()

    def rows(r, c, seed, pad=0, off=0):
        # every tensor ends where its memory ends: what is read behind it is not its own
        flat = inputs.normal((max((r - 1) * (c + pad) + c, 1) + off,), 1.0, seed, DEV)
        return flat[off:].as_strided((r, c), (c + pad, 1), off)

    def ints(r, c, seed, pad=0, off=0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        flat = torch.randint(-128, 128, ((r - 1) * (c + pad) + c + off,), generator=g, device=DEV, dtype=torch.int8)
        return flat.as_strided((r, c), (c + pad, 1), off)

    # the product: every kernel, aligned and not, edges inside tiles and 16-byte units
    seed = 0
    for M, N, K in ((1, 1, 1), (1, 37, 530), (2, 130, 96), (5, 33, 67), (16, 129, 640), (31, 200, 131), (70, 260, 1300),
                    (130, 129, 2049), (300, 515, 257)):
        for pad, off in ((0, 0), (5, 0), (16 - K % 16, 0), (16 - K % 16, 3)):
            seed += 1
            a, b = ints(M, K, seed, pad, off), ints(N, K, 1000 + seed, pad, off)
            sa, sb, bias = (inputs.normal((n,), 1.0, 2000 + seed + i, DEV) for i, n in enumerate((M, N, N)))
            for cfg in range(rp.gemm_i8_config_count()):
                for dt, pitch in ((torch.float32, 0), (torch.float16, 3), (torch.bfloat16, 0)):
                    C = torch.zeros((M - 1) * (N + pitch) + N, dtype=dt, device=DEV)
                    rp.gemm_i8(a, b.t(), sa, sb, out=C.as_strided((M, N), (N + pitch, 1)), bias=bias if pitch else None,
                               config=cfg)
                    done("i8_%d_%d_%s" % (seed, cfg, dt), C)
    # rows in 8 bits, and the backward operators that read them
    for r, c in ((1, 1), (3, 33), (9, 260), (40, 1023), (33, 2048), (5, 8200), (2, 33000), (1100, 36)):
        for group in (0, 32, 256):
            for pad, off in ((0, 0), (3, 1)):
                seed += 1
                name = "rows_%d_%d_%d_%d" % (r, c, group, pad)
                x, u, dy, res = (rows(r, c, 3000 + 4 * seed + i, pad, off) for i in range(4))
                q, s = rp.quantize_rows(x, group=group)
                qu, su = rp.quantize_rows(u.to(torch.bfloat16), group=group)
                done(name + "_q", q, s, qu, su)
                done(name + "_v", rp.dequantize_rows(q, s, group=group),
                     rp.dequantize_rows(qu, su, group=group, dtype=torch.float16))
                h = torch.empty(r, c, device=DEV)
                done(name + "_g", *rp.swiglu_backward_i8(q, s, qu, su, dy, group=group, h=h), h)
                gamma = inputs.normal((c,), 1.0, 5000 + seed, DEV)
                done(name + "_n", *rp.rmsnorm_backward_i8(q, s, gamma, 1e-5, dy, group=group, res=res, h=h), h)
    # the block edge, forward and backward, with every set of operands; long sums
    for r, c in ((1, 1), (6, 33), (4, 300), (6, 700), (34, 1023), (66, 2048), (6, 4100), (4, 8192), (4, 8193), (2, 33000),
                 (33792, 4)):
        for pad, off in ((0, 0), (3, 1)):
            for gates in (0, 1, 2):
                for post in (False, True):
                    seed += 1
                    x, f, dy, dh = (rows(r, c, 6000 + 4 * seed + i, pad, off) for i in range(4))
                    g = None if gates == 0 or r % gates else rows(gates, c, 9000 + seed, pad, off)
                    pre, p = inputs.normal((c,), 1.0, 9500 + seed, DEV), inputs.normal((c,), 1.0, 9600 + seed, DEV)
                    kw = dict(post_gain=p if post else None, gate=g, alpha=0.5)
                    name = "edge_%d_%d_%d_%d_%d" % (r, c, pad, gates, post)
                    y, h = rp.rmsnorm_residual(x, f, pre, 1e-5, **kw)
                    done(name, y, h)
                    done(name + "_b", *rp.rmsnorm_residual_backward(dy, dh, y, f, pre, 1e-5, **kw))
                    if post:
                        done(name + "_y", rp.rmsnorm_residual(x, f, None, 1e-5, **kw)[0],
                             *rp.rmsnorm_residual_backward(dy, None, None, f, None, 1e-5, **kw))
    done("colsum", rp.colsum(rows(33793, 7, 1, 2, 1)))
    return out


if __name__ == "__main__":
    import verifiable_repops_gemm_gb300 as rp
    from verifiable_repops_gemm_gb300 import _capi
    _capi.load(sys.argv[1])
    assert "-DREPOPS_DEBUG_BOUNDS" in rp.version(), rp.version()
    res = workloads(rp)
    np.savez(sys.argv[2], **res)
    print("checked run ok:", len(res), "results")
