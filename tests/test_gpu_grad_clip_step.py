"""GradClip with the optimizer step: the norm alone, which sbl_adamw_step clips by, and the clip in place,
after which it must not clip again."""
import pytest
import torch

import synth

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("max_norm", [0.25, 1e6])
def test_norm_and_clip_give_the_same_optimizer_step(lib, max_norm):
    """g * c is one fp32 product with one factor, in the clip or in the update: the same bits of W, its moments
    and its ternary weight."""
    from semi_structured_sparsity_step_b200.layer import GradClip, SparseBitLinearLayer
    d_out, d_in = 136, 272
    results = []
    for clip_in_place in (False, True):
        dw, m, v = (t.cuda() for t in synth.optimizer_state(d_out, d_in, seed=43, g_std=1.0))
        L = SparseBitLinearLayer(synth.trimodal_weight(d_out, d_in, seed=43).cuda(), 6, 8, keep_mask=True)
        other = torch.randn(777, generator=synth.gen(43, 9)).to(torch.bfloat16).cuda()
        C = GradClip([dw, other])
        C.clip(max_norm) if clip_in_place else C.norm_only()
        lib.sbl_adamw_step(L.W, None, dw, m, v, d_out, d_in, 6, 8, 1e-3, 0.9, 0.95, 1e-5, 0.1, 1, C.grad_sqnorm, max_norm,
                           L.W_eff, L.W_eff_bf16, L.mask_bits, L.gamma, None, L.ws, L.ws_bytes)
        lib.sbl_check()
        assert (C.norm.item() > max_norm) == (max_norm == 0.25)
        results.append([L.W, m, v, L.W_eff, L.gamma, C.sumsq])
    assert all(torch.equal(a, b) for a, b in zip(*results))
