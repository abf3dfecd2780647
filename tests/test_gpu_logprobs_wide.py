"""Token log probabilities of rows that several CTAs of a cluster share, of more
segments than the cluster's warps and of more blocks than are ranked at once, up to
the most columns there may be: bit for bit against the step-by-step definition, and
the same bits however many rows there are."""
import numpy as np
import pytest
import torch

import logprobs_ref as ref
from test_gpu_logprobs import DEV, DT, check, host, logits, same, some_targets

pytestmark = pytest.mark.gpu


def shape(cols, rows, sms):
    """(warps a CTA, CTAs a row) of the rule that shares a row's segments."""
    segments = -(-cols // 4096)
    warps, ctas = 4 if segments >= 4 else 1, 1
    while warps < 8 and warps < segments and rows * warps < 32 * sms:
        warps *= 2
    while ctas < 8 and ctas * warps < segments and rows * warps * ctas < 32 * sms:
        ctas *= 2
    if ctas == 1:
        warps = -(-segments // -(-segments // warps))
    return warps, ctas


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("cols", [70001, 100003, 300007])
def test_every_cluster_size_gives_a_row_the_same_bits(rp, kind, cols):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    counts = [1, 2 * sms + 8, 4 * sms + 50, 9 * sms] if cols < 300000 else [1, 2, sms // 2, sms + 8, 4 * sms + 50]
    shapes = {shape(cols, n, sms) for n in counts}
    assert {c for _, c in shapes} == ({1, 2, 4} if cols < 300000 else {1, 4, 8})
    rows = max(counts)
    x, t = logits(rows, cols, kind, cols), some_targets(rows, cols, 6)
    x[:, 20000:20100] = -np.inf
    whole = rp.token_logprobs(x, t, top=7)
    for n in counts:
        part = rp.token_logprobs(x[:n], t[:n], top=7)
        for a, b in zip(part, whole):
            assert torch.equal(a, b[:n]), n
    pick = torch.tensor([0, 1, rows // 2, rows - 1])
    want = ref.forward(host(x[pick]), host(t[pick]), 1.0, 7)
    for a, w in zip(whole, want):
        assert same(host(a[pick]), w) if a.is_floating_point() else np.array_equal(host(a[pick]), w)


@pytest.mark.parametrize("kind,pad,off", [("f32", 0, 0), ("f32", 2, 1), ("bf16", 0, 0), ("bf16", 5, 3), ("f16", 1, 0)])
@pytest.mark.parametrize("top", [1, 20, 32])
def test_more_blocks_than_are_ranked_at_once(rp, kind, pad, off, top):
    cols = 400003                                            # 391 blocks of 1024, 98 segments
    x = logits(2, cols, kind, 11 + top, pad, off)
    x[1, 1000:390000] = -np.inf
    x[1, [cols - 1, 399000]] = 30.0
    check(rp, x, torch.tensor([cols - 1, 5], device=DEV), 0.8, top)


@pytest.mark.parametrize("cols,kind,rows,pad,off", [(7_000_001, "f32", 2, 2, 1), (8_388_608, "f16", 1, 0, 0),
                                                    (16_384_000, "bf16", 1, 0, 0), (16_383_999, "bf16", 1, 0, 3)])
def test_up_to_the_most_columns(rp, cols, kind, rows, pad, off):
    """Above 6.6 million columns a row's sums and maxima pass 48 KB of shared memory."""
    x = logits(rows, cols, kind, 13, pad, off)
    x[0, cols - 1] = 25.0
    t = torch.full((rows,), cols - 1, device=DEV)
    t[0] = cols // 3
    got = check(rp, x, t, 1.0, 5)
    assert host(got.top_ids)[0, 0] == cols - 1
    dl, de = (torch.randn(rows, generator=torch.Generator(device=DEV).manual_seed(4 + i), device=DEV) for i in (0, 1))
    d = rp.token_logprobs_backward(x, t, got.stats, dl, de)
    want = ref.backward(host(x), host(t), host(got.stats), host(dl), host(de), 1.0)
    assert same(host(d), host(torch.from_numpy(want).to(DT[kind])))


@pytest.mark.parametrize("kind,cols", [("f32", 5), ("bf16", 130)])
def test_more_rows_than_a_grid_is_high(rp, kind, cols):
    """The gradient's rows past 65535 are a block's second ones."""
    rows = 140001
    x, t = logits(rows, cols, kind, 3), some_targets(rows, cols, 4)
    got = rp.token_logprobs(x, t, top=2)
    dl = torch.randn(rows, generator=torch.Generator(device=DEV).manual_seed(5), device=DEV)
    d = rp.token_logprobs_backward(x, t, got.stats, dl, None)
    pick = torch.tensor([0, 1, 65534, 65535, 65536, 131069, 131070, rows - 1], device=DEV)
    want = ref.forward(host(x[pick]), host(t[pick]), 1.0, 2)
    for a, w in zip(got, want):
        assert same(host(a[pick]), w) if a.is_floating_point() else np.array_equal(host(a[pick]), w)
    want = ref.backward(host(x[pick]), host(t[pick]), host(got.stats[pick]), host(dl[pick]), None, 1.0)
    assert same(host(d[pick]), host(torch.from_numpy(want).to(DT[kind])))
    # and every row by elementary operations: probabilities of at most one, a few roundings
    p = torch.softmax(x.float(), 1)
    w = torch.where(t < 0, torch.zeros_like(dl), dl)[:, None]
    plain = -p * w
    plain.scatter_add_(1, t.clamp_min(0)[:, None], w)
    half = {"f32": 0.0, "bf16": 2.0 ** -8}[kind]
    assert ((d.float() - plain).abs() <= plain.abs() * half + w.abs() * 2.0 ** -19 + 1e-37).all()
