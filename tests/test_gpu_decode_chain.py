"""One decode step of a beam search, the operators one after another as a serving loop runs them: block-FP8
projection, gated delta rule over the beams' states, block-FP8 projection, MoE layer, FP8 LM head, selection over
beams and vocabulary, reorder of the states.  Every operator is checked against its own 64-bit oracle on the inputs
it was given, over two steps; then the step is captured into a graph and replayed to the same bits.
"""
import numpy as np
import pytest
import torch

import oracle
import oracle.beam_ref as B
import oracle.delta_ref as D
import oracle.fp8_linear_ref as F
import weight_only_int4_fp32_b200 as lm
import workloads
from tests.parity import bits, compare

pytestmark = pytest.mark.gpu
DEV = "cuda"
W, H, HEADS, DIM, VOCAB = 4, 2560, 4, 128, 1000
EOS = 3


def linear_weights(N, K, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    w = torch.randn(N, K, generator=g, device=DEV) * 40.0
    s = torch.rand(-(-N // 128), -(-K // 128), generator=g, device=DEV) * 5e-4 + 2e-4
    return w.clamp(-448, 448).to(torch.float8_e4m3fn), s


def check_linear(y, x, codes, scales):
    """The bound of the linear layer's own tests: (25 + blocks) u of the magnitudes, and half a bf16 step."""
    want, mag = F.linear(x.float().cpu().numpy(), codes.view(torch.uint8).cpu().numpy(), scales.cpu().numpy())
    tol = (25 + scales.shape[1]) * 2.0**-24 * mag + 2.0**-8 * np.abs(want) + 1e-37
    assert (np.abs(y.double().cpu().numpy() - want) <= tol).all()


class Step:
    def __init__(self):
        self.w_in, self.w_out = linear_weights(3 * HEADS * DIM, H, 1), linear_weights(H, HEADS * DIM, 2)
        self.proj = lm.BlockFP8Linear(*self.w_in, max_tokens=W)
        self.out = lm.BlockFP8Linear(*self.w_out, max_tokens=W)
        self.delta = lm.GatedDeltaRule(HEADS, HEADS, DIM, DIM, max_tokens=W, max_seqs=W)
        lw = workloads.layer_weights(32, seed=0, device="cpu")
        self.host = lw.host_arrays()
        self.moe = lm.MoELayer({k: (None if v is None else v.to(DEV)) for k, v in lw.tensors().items()}, top_k=8, max_tokens=W)
        self.head = lm.LMHeadFP8(workloads.lm_head_weights(VOCAB, H, seed=3, device="cpu").to(DEV))
        self.beams = lm.BeamSearch(1, W, VOCAB)
        self.embed = torch.stack([workloads.tokens(1, seed=t, device="cpu")[0] for t in range(64)]).to(DEV)
        g = torch.Generator(device=DEV).manual_seed(5)
        self.g = -torch.rand(W, 1, HEADS, DIM, generator=g, device=DEV)
        self.beta = torch.rand(W, 1, HEADS, generator=g, device=DEV)
        self.slots = torch.tensor([3, 0, 4, 1], dtype=torch.int32, device=DEV)  # of a pool of five

    def begin(self):
        g = torch.Generator(device=DEV).manual_seed(6)
        state = 0.3 * torch.randn(5, HEADS, DIM, DIM, generator=g, device=DEV)
        scores = torch.tensor([[0.0, -0.1, -0.2, -0.3]], device=DEV)
        return dict(state=state, tokens=torch.arange(W, dtype=torch.int32, device=DEV).view(1, W), scores=scores,
                    finished=torch.zeros(1, W, dtype=torch.bool, device=DEV))

    def run(self, s):
        """One step in place on s; returns what every operator was given and gave."""
        x = self.embed[(s["tokens"].clamp(min=0) % 64).view(W).long()]
        qkv = self.proj(x)
        q, k, v = (t.view(W, 1, HEADS, DIM) for t in qkv.split(HEADS * DIM, 1))
        a = self.delta.step(q, k, v, self.g, self.beta, s["state"], slots=self.slots)
        y = self.out(a.view(W, HEADS * DIM))
        z, idx, wt = self.moe(y, return_routing=True)
        logits = self.head(z)
        tokens, parents, scores, finished = self.beams.select(logits, s["scores"], s["finished"], EOS)
        stepped = s["state"].clone()
        self.beams.reorder(s["state"], parents, slots=self.slots.view(1, W))
        seen = dict(x=x, qkv=qkv, q=q, k=k, v=v, a=a, y=y, z=z, idx=idx, wt=wt, logits=logits, parents=parents, stepped=stepped,
                    scores_in=s["scores"].clone(), finished_in=s["finished"].clone(), tokens=tokens, scores=scores,
                    finished=finished)
        s["tokens"].copy_(tokens), s["scores"].copy_(scores), s["finished"].copy_(finished)
        return seen


def test_two_steps_of_a_beam_search():
    step = Step()
    s = step.begin()
    np64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    for _ in range(2):
        before = s["state"].clone()
        r = step.run(s)
        torch.cuda.synchronize()
        check_linear(r["qkv"], r["x"], *step.w_in)
        for i, slot in enumerate(step.slots.tolist()):
            x = [np64(t[i]) for t in (r["q"], r["k"], r["v"], step.g, step.beta)]
            want, states = D.rule(*x, np64(before[slot]), DIM**-0.5)
            eo, es = D.step_bound(*x, np64(before[slot]), DIM**-0.5)
            assert (np.abs(np64(r["a"][i]) - want) <= eo + 2.0**-8 * (np.abs(want) + eo)).all()
            err = np.linalg.norm(np64(r["stepped"][slot]) - states[-1], axis=1)
            assert (err <= es[-1] + 2.0**-24 * np.linalg.norm(states[-1], axis=1)).all()
        check_linear(r["y"], r["a"].view(W, -1), *step.w_out)
        compare(oracle.moe_layer(bits(r["y"].cpu()), step.host, 8), r["z"], r["idx"], r["wt"], 8, "chain")
        wt, wp, ws, wd = B.select(r["logits"].cpu().numpy().reshape(1, W, VOCAB), r["scores_in"].cpu().numpy(),
                                  r["finished_in"].cpu().numpy(), EOS)
        assert np.array_equal(r["tokens"].cpu().numpy(), wt) and np.array_equal(r["parents"].cpu().numpy(), wp)
        assert np.array_equal(r["finished"].cpu().numpy(), wd)
        par = r["parents"][0].long()
        assert torch.equal(s["state"][step.slots.long()], r["stepped"][step.slots.long()[par]])
        assert torch.equal(s["state"][2], before[2])  # the slot that no beam holds
    # the same two steps from a captured graph
    eager, replay = s, step.begin()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.run(replay)
    start = step.begin()
    for k in start:
        replay[k].copy_(start[k])
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for k in eager:
        assert torch.equal(eager[k], replay[k]), k
    for op in (step.proj, step.out, step.delta, step.moe, step.head):
        assert op.status() == lm.LING_MOE_OK
