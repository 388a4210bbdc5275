"""The block norm between two decode products, back to back on one stream: the second product is set up, and
streams its weights, while the norm still writes the codes that it reads."""
import pytest
import torch

import synth

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("variant", [0, 1, 2])
@pytest.mark.parametrize("layout", ["dense2", "6:8"])
@pytest.mark.parametrize("batch", [1, 4, 16])
def test_back_to_back_is_what_one_call_at_a_time_gives(lib, batch, layout, variant):
    d0, d1, d2, rounds = 512, 2048, 1024, 24
    dev = dict(device="cuda")
    gamma = torch.tensor([0.02], **dev)
    gain = torch.ones(d1, dtype=torch.bfloat16, **dev)

    def packed(d_out, d_in, seed):
        W = synth.trimodal_weight(d_out, d_in, seed=seed).cuda()
        weff, g = torch.empty(d_out, d_in, dtype=torch.int8, **dev), torch.empty(1, **dev)
        n = lib.sbl_mask_quant_workspace_bytes(d_out, d_in)
        lib.sbl_mask_quant(W, d_out, d_in, 6, 8, weff, None, None, g, torch.empty(n, dtype=torch.uint8, **dev), n)
        size = lib.sbl_dense2_bytes(d_out, d_in) if layout == "dense2" else lib.sbl_packed_bytes(d_out, d_in, 6, 8)
        out = torch.empty(size, dtype=torch.uint8, **dev)
        if layout == "dense2":
            lib.sbl_pack_dense2(weff, d_out, d_in, out, size)
        else:
            lib.sbl_pack(weff, d_out, d_in, 6, 8, out, size)
        torch.cuda.synchronize()
        return out

    w1, w2 = packed(d1, d0, 1), packed(d2, d1, 2)
    xs = [synth.activations(batch, d0, seed=10 + k).cuda() for k in range(rounds)]
    hs = [synth.activations(batch, d1, seed=50 + k).cuda() for k in range(rounds)]
    xq, am, y = torch.empty(batch, d0, dtype=torch.int8, **dev), torch.empty(batch, **dev), torch.empty(batch, d1, **dev)
    h, q2, am2 = torch.empty_like(hs[0]), torch.empty(batch, d1, dtype=torch.int8, **dev), torch.empty(batch, **dev)

    def product(w, codes, amax, out, d_in, d_out):
        group = [(w, codes, amax, gamma, out, d_in, d_out)]
        if layout == "dense2":
            lib.sbl_gemv_dense2_group(group, batch)
        else:
            lib.sbl_gemv_packed_group(group, batch, 6, 8)

    def run(between):
        outs = torch.full((rounds, batch, d2), -1.0, **dev)
        q2.fill_(1)
        am2.fill_(1.0)
        for k in range(rounds):
            lib.sbl_act_quant(xs[k], batch, d0, xq, am)
            between()
            product(w1, xq, am, y, d0, d1)
            between()
            lib.sbl_block_norm(y, hs[k], gain, None, 0, 1.0, gain, 1e-6, batch, d1, 0, h, None, q2, am2, None)
            between()
            product(w2, q2, am2, outs[k], d1, d2)
            between()
        lib.sbl_check()
        return outs

    lib.sbl_set_gemv_variant(variant)
    try:
        want = run(torch.cuda.synchronize)
        assert not torch.equal(want[0], want[1])
        for _ in range(4):
            assert torch.equal(run(lambda: None), want)
    finally:
        lib.sbl_set_gemv_variant(0)
