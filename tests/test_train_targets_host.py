"""What a training step takes as targets: int64 tokens, and no other whole numbers."""
import pytest
import torch


def test_targets_of_another_integer_type_are_refused():
    """int32 targets are no upstream gradient, also where a row of them would spread over
    the model's width."""
    from verifiable_repops_gemm_gb300 import decoder, train
    cfg = decoder.DecoderConfig(d=32, heads=2, kv_heads=2, ffn=32, seq_len=8)
    model = train.Model(cfg, 1, "cpu", vocab=40)
    was = model.theta.clone()
    for kind in (torch.int32, torch.int16, torch.uint8, torch.bool):
        for tokens in (32, 8):
            with pytest.raises(ValueError, match="int64"):
                train.train_step(model, [(b"did:a", torch.zeros(tokens, 32), torch.ones(tokens).to(kind))], 0.1, None)
    assert torch.equal(model.theta, was)
