"""A verifiable data-parallel training step on one GPU, every step a library
call: contributors' gradients through a decoder model, the fixed-order
aggregation, the update and the commitment.

"Zoo Per-LLM Chain Soundness" §2 (Definition "Aggregation rule": the average of
the contributors' gradients; Lemma "Order independence within a batch"), §5
("Ordering subroutine": contributors sorted by DID bytes, the left fold;
"Update step": theta_t = theta_{t-1} - eta * gbar_t), §1 and §6 (the model
state committed as a Merkle root); "Verde与RepOps" §4.3 (Llama-style training
as the workload).

theta is one flat float32 vector holding every layer's weights, each at a
16-byte-aligned offset in a fixed order (the gaps stay +0); the Merkle root
commits exactly its bytes.  A contributor's gradient is a flat vector of the
same layout: forward through the layers keeping their activations, then the
backward pass from the contributor's upstream gradient.  A step sorts the
contributors' DIDs, folds their gradients in that order into the mean, applies
SGD (or AdamW, whose moments are committed alike) to theta in place and returns
the root of the new theta -- the same bits whatever order the gradients were
computed in.

With a vocabulary the model ends in a norm and a product to logits, and a
contribution may hold target tokens in the place of an upstream gradient: the loss
is the mean of their negative log probabilities (token_logprobs).
"""
import math

import torch

from . import (ADAMW_GROUP, adamw, colsum, decoder, fixed_order_mean_sgd, gemm, merkle_sha256, rmsnorm_backward,
               rmsnorm_rows, sort_ids, token_logprobs, token_logprobs_backward)


def layout(cfg: decoder.DecoderConfig, layers: int, vocab: int = 0):
    """[(layer, key, offset, shape)] and the total length of theta: layer by
    layer, each layer's weights in `decoder.weight_shapes` order, then with a
    vocabulary the last norm's gain and the logits' weights (as layer `layers`),
    every tensor starting at a multiple of 4 elements (16 bytes: TMA-describable)."""
    out, off = [], 0
    shapes = decoder.weight_shapes(cfg)
    for layer in range(layers + (vocab > 0)):
        if layer == layers:
            shapes = {"g_out": (cfg.d,), "w_out": (cfg.d, vocab)}
        for key, shape in shapes.items():
            n = 1
            for s in shape:
                n *= s
            out.append((layer, key, off, shape))
            off += (n + 3) // 4 * 4
    return out, off


class Model:
    """`layers` decoder layers, and with a vocabulary the logits' norm and weights
    (weights[layers]), whose weights are views into one flat theta."""

    def __init__(self, cfg: decoder.DecoderConfig, layers: int, device, seed: int = 0, vocab: int = 0):
        self.cfg, self.layers, self.vocab = cfg, layers, vocab
        self.slots, n = layout(cfg, layers, vocab)
        self.theta = torch.zeros(n, dtype=torch.float32, device=device)
        self.weights = self.views(self.theta)
        for layer in range(layers):
            init = decoder.init_weights(cfg, seed + layer, device)
            for key, v in init.items():
                self.weights[layer][key].copy_(v)
        if vocab:
            gen = torch.Generator(device=device).manual_seed(seed + layers)
            self.weights[layers]["g_out"].fill_(1.0)
            self.weights[layers]["w_out"].copy_(torch.randn(cfg.d, vocab, generator=gen, device=device) * 0.02)

    def views(self, flat):
        """Per layer, {key: view} of a flat buffer with theta's layout."""
        vs = [{} for _ in range(self.layers + (self.vocab > 0))]
        for layer, key, off, shape in self.slots:
            n = 1
            for s in shape:
                n *= s
            vs[layer][key] = flat[off:off + n].view(shape)
        return vs

    def gradient_buffer(self):
        """A flat gradient vector (its alignment gaps stay +0)."""
        return torch.zeros_like(self.theta)


class Workspace:
    """Buffers one contributor's forward and backward reuse.  checkpoint_bits=8
    keeps the layers' activations in 8 bits (decoder.activations): every
    contributor and every verifier must choose the same, as the gradients' bits
    depend on it."""

    def __init__(self, model: Model, tokens: int, device, checkpoint_bits: int = 32):
        cfg = model.cfg
        self.saved = [decoder.activations(cfg, tokens, device, checkpoint_bits) for _ in range(model.layers)]
        self.fwd = decoder.workspace(cfg, tokens, device)
        self.bwd = decoder.backward_workspace(cfg, tokens, device, checkpoint_bits)
        self.h = torch.empty(tokens, cfg.d, dtype=torch.float32, device=device)
        self.d = torch.empty(tokens, cfg.d, dtype=torch.float32, device=device)
        if model.vocab:
            self.logits = torch.empty(tokens, model.vocab, dtype=torch.float32, device=device)
            self.t = torch.empty(tokens, cfg.d, dtype=torch.float32, device=device)


def _forward(model: Model, x, ws: Workspace):
    ws.h.copy_(x)
    for layer in range(model.layers):
        decoder.forward(ws.h, model.weights[layer], model.cfg, work=ws.fwd, save=ws.saved[layer])


def _backward(model: Model, gviews, ws: Workspace):
    d = ws.d
    for layer in reversed(range(model.layers)):
        d, _ = decoder.backward(d, model.weights[layer], model.cfg, ws.saved[layer], work=ws.bwd, grads=gviews[layer])


def contributor_gradient(model: Model, x, dy, grad_flat, ws: Workspace):
    """grad_flat <- the gradient of the model's parameters for input x and
    upstream gradient dy (both T x d: of the last layer's output, so that a
    vocabulary's norm and weights get 0); returns grad_flat."""
    _forward(model, x, ws)
    ws.d.copy_(dy)
    gviews = model.views(grad_flat)
    for g in gviews[model.layers:]:
        for v in g.values():
            v.zero_()
    _backward(model, gviews, ws)
    return grad_flat


def token_gradient(model: Model, x, targets, grad_flat, ws: Workspace):
    """grad_flat <- the gradient, for input x (T x d), of the mean negative log
    probability of targets (int64, T; a negative one is no target) under a model
    with a vocabulary; returns (grad_flat, the targets' log probabilities)."""
    if not model.vocab:
        raise ValueError("the model has no vocabulary to take targets from")
    cfg, out = model.cfg, model.weights[model.layers]
    _forward(model, x, ws)
    h = rmsnorm_rows(ws.h, out["g_out"], cfg.eps, out=ws.t)
    logits = gemm(h, out["w_out"], out=ws.logits)
    r = token_logprobs(logits, targets)
    count = (targets >= 0).sum().clamp_min(1).to(torch.float32)
    weight = (-1.0 / count).expand(targets.numel()).contiguous()
    dlogits = token_logprobs_backward(logits, targets, r.stats, weight, out=logits)
    gviews = model.views(grad_flat)
    g = gviews[model.layers]
    gemm(h.t(), dlogits, out=g["w_out"])
    dh = gemm(dlogits, out["w_out"].t(), out=ws.t)
    _, terms = rmsnorm_backward(ws.h, out["g_out"], cfg.eps, dh, dx=ws.d)
    colsum(terms, out=g["g_out"])
    _backward(model, gviews, ws)
    return grad_flat, r.logp


class AdamW:
    """AdamW over a model's parameters (adamw), one tensor a weight, decaying
    matrices alone; its moments lie in flat buffers of theta's layout (bits=8: a
    byte each, with scale bytes for every 128 elements of a weight)."""

    def __init__(self, model: Model, lr: float, betas=(0.9, 0.95), eps: float = 1e-8, weight_decay: float = 0.1,
                 bits: int = 32, seed: int = 0):
        if bits not in (32, 8):
            raise ValueError("bits must be 32 or 8")
        self.model, self.lr, self.betas, self.eps, self.seed, self.steps = model, lr, betas, eps, seed, 0
        self.spans = [(off, math.prod(shape)) for _, _, off, shape in model.slots]
        self.decay = [weight_decay if len(shape) > 1 else 0.0 for _, _, _, shape in model.slots]
        n, dev = model.theta.numel(), model.theta.device
        kind = torch.float32 if bits == 32 else torch.uint8
        self.state = {k: torch.zeros(n, dtype=kind, device=dev) for k in ("m", "v")}
        views = {k: self._slots(t) for k, t in self.state.items()}
        if bits == 8:
            groups = [-(-k // ADAMW_GROUP) for _, k in self.spans]
            for name in ("m_scales", "v_scales"):
                self.state[name] = torch.zeros(sum(groups), dtype=torch.uint8, device=dev)
                views[name] = list(self.state[name].split(groups))
        self.views = views

    def _slots(self, flat):
        return [flat[off:off + n] for off, n in self.spans]

    def step(self, grads, order) -> None:
        """One step of theta from the contributors' flat gradients, folded in `order`."""
        adamw(self._slots(self.model.theta), [self._slots(g) for g in grads], step=self.steps + 1, lr=self.lr,
              betas=self.betas, eps=self.eps, weight_decay=self.decay, order=order, seed=self.seed, **self.views)
        self.steps += 1

    def roots(self):
        """The Merkle root of each of the moments' buffers.  A replay of later steps has to
        start from these and theta's, and from what they do not hold: `steps` (the bias
        corrections and the dither hang on it) and the constructor's arguments.  An
        optimiser built alike goes on where `state` is copied in and `steps` set."""
        return {name: merkle_sha256(t) for name, t in self.state.items()}


def train_step(model: Model, contributions, eta: float, ws: Workspace, grads=None, optimizer: AdamW = None):
    """contributions: [(did bytes, x, dy)], or with a vocabulary [(did bytes, x,
    int64 targets)], in any order.  Computes every contributor's gradient, folds
    them in DID order into the mean, applies SGD with eta (or the optimizer's step)
    to theta in place and returns (root of the new theta, the order)."""
    if model.vocab and any(not d.is_floating_point() and d.dtype != torch.int64 for _, _, d in contributions):
        raise ValueError("targets must be int64")    # not an upstream gradient of whole numbers
    if grads is None:
        grads = [model.gradient_buffer() for _ in contributions]
    for (did, x, d), g in zip(contributions, grads):
        if d.dtype == torch.int64:
            token_gradient(model, x, d, g, ws)
        else:
            contributor_gradient(model, x, d, g, ws)
    order = sort_ids([did for did, _, _ in contributions])
    if optimizer is None:
        fixed_order_mean_sgd(grads, order, eta, model.theta)
    else:
        optimizer.step(grads, order)
    return merkle_sha256(model.theta), order
