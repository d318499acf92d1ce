"""A handle that is created while its weights are still being written, on the default stream or another one, holds
the weights as they will be: create waits for the device first."""
import pytest
import torch

import weight_only_int4_fp32_b200 as lm
import workloads

pytestmark = pytest.mark.gpu
DEV = "cuda"


def late(tensors, stream):
    """Buffers that get `tensors` only some tens of milliseconds later, on `stream`."""
    bufs = [None if t is None else torch.zeros_like(t) for t in tensors]
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(60_000_000)  # clock cycles
        for b, t in zip(bufs, tensors):
            if b is not None:
                b.copy_(t)
    return bufs


@pytest.mark.parametrize("side", [False, True])
def test_create_waits_for_its_weights(side):
    st = torch.cuda.Stream() if side else torch.cuda.current_stream()
    x = workloads.tokens(2, seed=1, device="cpu").to(DEV)
    w = {k: (None if v is None else v.to(DEV)) for k, v in workloads.layer_weights(32, seed=0, device="cpu").tensors().items()}
    want = lm.MoELayer(w, top_k=8, max_tokens=2).forward(x)
    layer = lm.MoELayer(dict(zip(w, late(list(w.values()), st))), top_k=8, max_tokens=2)
    assert torch.equal(layer.forward(x), want)

    head = workloads.lm_head_weights(1000, 2560, seed=3, device="cpu").to(DEV)
    want = lm.LMHeadFP8(head).forward(x)
    assert torch.equal(lm.LMHeadFP8(late([head], st)[0]).forward(x), want)

    g = torch.Generator(device=DEV).manual_seed(2)
    codes = (torch.randn(256, 2560, generator=g, device=DEV) * 60).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    scales = torch.rand(2, 20, generator=g, device=DEV)
    want = lm.BlockFP8Linear(codes, scales, max_tokens=2).forward(x)
    assert torch.equal(lm.BlockFP8Linear(*late([codes, scales], st), max_tokens=2).forward(x), want)
