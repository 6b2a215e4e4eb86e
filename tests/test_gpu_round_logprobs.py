"""Round.emitted_logprobs into buffers of the caller, which a captured round replays."""
import pytest
import torch

from tree_speculative_decoding_02_gb300 import ddt, synth
from tree_speculative_decoding_02_gb300.round import Round

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("temperature", [0.0, 0.8])
def test_given_buffers(temperature):
    cfg = dict(synth.WORKLOADS[1], V=3000, budget=24, B=3, temperature=temperature, dtype=torch.bfloat16, Lf=0, Lg=0)
    r = Round(cfg, device="cuda", workload=1)
    r.step()
    want = r.emitted_logprobs(top_n=4)
    ws = ddt.token_logprobs_workspace(r.target_logits, r.walk["emitted"], top_n=4)
    out = {k: torch.full_like(v, -9) for k, v in want.items()}
    before = torch.cuda.memory_stats()["allocation.all.allocated"]
    got = r.emitted_logprobs(top_n=4, out=out, workspace=ws)
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == before
    assert all(got[k] is out[k] and torch.equal(out[k], want[k]) for k in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r.emitted_logprobs(top_n=4, out=out, workspace=ws)
    for v in out.values():
        v.fill_(-9)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out[k], want[k]) for k in want)
