"""AdamW given its tensors by iterators, once or from several contributors."""
import pytest
import torch

from test_gpu_adamw import HYPER, problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("k", [1, 3])
def test_iterators_are_lists(rp, bits, k):
    sizes = [300, 0, 5, 4097]
    how = dict(step=3, lr=1e-3, seed=1, **HYPER)
    theta, grads, st = problem(sizes, k, "bf16", 17, bits=bits)
    other = [torch.nn.Parameter(t.clone(), requires_grad=False) for t in theta]
    st2 = {n: [t.clone() for t in ts] for n, ts in st.items()}
    rp.adamw(theta, grads if k > 1 else grads[0], **st, weight_decay=[0.1, 0.0, 0.0, 0.2], **how)
    given = (iter(g) for g in grads) if k > 1 else iter(grads[0])
    rp.adamw(torch.nn.ParameterList(other).parameters(), given, **{n: iter(ts) for n, ts in st2.items()},
             weight_decay=iter([0.1, 0.0, 0.0, 0.2]), **how)
    assert all(torch.equal(a, b) for a, b in zip(theta, other))
    assert all(torch.equal(a, b) for n in st for a, b in zip(st[n], st2[n]))


def test_one_tensor_and_none(rp):
    theta, grads, st = problem([77], 2, "f32", 3)
    one, st1 = theta[0].clone(), {n: t[0].clone() for n, t in st.items()}
    rp.adamw(theta, grads, **st, step=1, lr=1e-3)
    rp.adamw(one, [[g[0]] for g in grads], **st1, step=1, lr=1e-3)
    assert torch.equal(one, theta[0])
    rp.adamw(iter(()), iter(()), m=iter(()), v=iter(()), step=1, lr=1e-3)
    with pytest.raises(ValueError):
        rp.adamw(iter(theta), iter(()), m=iter(st["m"]), v=iter(st["v"]), step=1, lr=1e-3)
