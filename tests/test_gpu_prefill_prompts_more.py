"""ae_prefill_prompts under stream capture."""
import ctypes

import numpy as np
import pytest

from flow_matching_action_gb300 import synth

from .test_gpu_prefill_prompts import TINY, Prefill, bf16

pytestmark = pytest.mark.gpu


def test_first_prefill_inside_a_capture_is_refused_and_a_later_one_replays():
    """The first prefill builds the conditioning table (it allocates): refused while the stream captures,
    without breaking the capture.  After one outside, a captured prefill replays the same bits."""
    import torch

    from flow_matching_action_gb300 import ae
    d = TINY
    p = Prefill(d, synth.make_vlm_weights(d, 3), 4)
    ex, st = p.ex, torch.cuda.Stream()
    try:
        cu = [0, 3, 4]
        emb = bf16(np.random.default_rng(1).standard_normal((4, d.width)))
        pos = torch.tensor([0, 1, 2, 0], dtype=torch.int32, device="cuda")
        k = torch.zeros((d.layers, 4, d.kv_dim), dtype=torch.bfloat16, device="cuda")
        v, x = torch.zeros_like(k), torch.zeros(8, device="cuda")
        torch.cuda.synchronize()
        ae.ae_set_stream(ex.ctx, ctypes.c_void_p(st.cuda_stream))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            with pytest.raises(ae.AEError, match="outside of a capture") as e:
                ex.prefill_prompts(emb, cu, pos, k, v)
            assert e.value.status == -3  # AE_ERR_NOT_BOUND
            x.add_(1)
        graph.replay()
        torch.cuda.synchronize()
        assert (x == 1).all() and (k == 0).all()
        ex.prefill_prompts(emb, cu, pos, k, v)
        ex.synchronize()
        want = k.clone(), v.clone()
        assert (k != 0).any()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            ex.prefill_prompts(emb, cu, pos, k, v)
        for _ in range(2):
            k.zero_()
            v.zero_()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(k, want[0]) and torch.equal(v, want[1])
        ex.synchronize()
    finally:
        ex.close()
