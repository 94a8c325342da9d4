"""The delta rule's entries on a given stream, and their buffers' checks."""

import pytest
import torch

from workloads import make_case

pytestmark = pytest.mark.gpu


def problem(save=0):
    import chunkwise_delta_rule_gb300 as kda
    c = make_case(io="bf16", gate="channel", B=2, T=300, H=2, K=128, V=128, seed=91).to("cuda")
    return kda.make_problem(c.q, c.k, c.v, c.g, c.beta, gate="channel", initial_state=c.h0, save_policy=save), c


@pytest.mark.parametrize("name", ["chunk_fwd", "recurrent_fwd", "chunk_bwd", "chunk_bwd_saved"])
def test_a_given_stream_owns_what_the_call_allocates(name):
    """As for the layer operators: workspace and outputs of a call on a busy side stream lie neither in blocks that the
    current stream has freed but still writes, nor in blocks that its later tensors get."""
    import chunkwise_delta_rule_gb300 as kda
    save = int(name.endswith("saved"))
    p, c = problem(save)
    saved = kda.kda_chunk_fwd(p)[2]

    def call(st):
        if name == "chunk_fwd":
            return kda.kda_chunk_fwd(p, stream=st)
        if name == "recurrent_fwd":
            return kda.kda_recurrent_fwd(p, stream=st)
        return kda.kda_chunk_bwd(p, c.do, c.dht, saved=saved, stream=st)

    want = [t.clone() for t in call(None) if t is not None]
    torch.cuda.synchronize()
    sizes = [1 << b for b in range(9, 27)] + [4096 * i for i in range(1, 400, 7)]
    side, main = torch.cuda.Stream(), torch.cuda.current_stream()
    torch.cuda._sleep(40_000_000)
    late = [torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255) for n in sizes]
    del late
    got = call(side)                        # side does not wait for them
    side.synchronize()
    first = [t.clone() for t in got if t is not None]
    with torch.cuda.stream(side):
        torch.cuda._sleep(40_000_000)
    got = call(side)
    later = [torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255) for n in sizes]
    main.wait_stream(side)
    torch.cuda._sleep(40_000_000)
    second = [t.clone() for t in got if t is not None]
    del got                                 # still to be read
    with torch.cuda.stream(side):
        again = [torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255) for n in sizes]
    torch.cuda.synchronize()
    del later, again
    for got in (first, second):
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_host_buffers_are_refused():
    import chunkwise_delta_rule_gb300 as kda
    p, c = problem()
    ps, _ = problem(1)
    n = max(kda.kda_workspace_size(p, b) for b in (False, True))
    host = torch.empty(n, dtype=torch.uint8)
    with pytest.raises(ValueError, match="workspace must be"):
        kda.kda_chunk_fwd(p, workspace=host)
    with pytest.raises(ValueError, match="workspace must be"):
        kda.kda_chunk_bwd(p, c.do, c.dht, workspace=host)
    with pytest.raises(ValueError, match="do must be"):
        kda.kda_chunk_bwd(p, c.do.cpu(), c.dht)
    with pytest.raises(ValueError, match="ht must be"):
        kda.kda_recurrent_fwd(p, ht=c.h0.cpu())
    saved = torch.empty(kda.kda_saved_size(ps), dtype=torch.uint8)
    with pytest.raises(ValueError, match="saved must be"):
        kda.kda_chunk_fwd(ps, saved=saved)
    for bad in (None, saved[:16].cuda()):
        with pytest.raises(ValueError, match="saved buffer"):
            kda.kda_chunk_bwd(ps, c.do, c.dht, saved=bad)
