"""The allocating helpers of the training calls on a stream that is not the current one."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def msa():
    import __graft_entry__

    __graft_entry__.build_library()
    import block_sparse_attention_scores_gb300 as m

    return m


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
def test_helpers_allocate_on_the_stream_they_run_on(msa, raw):
    """Workspaces and outputs come from the side stream: they are neither taken from what the current stream still writes
    to, nor handed out to it while the side stream has the call to do."""
    import torch

    gen = torch.Generator().manual_seed(1)

    def normal(*shape):
        return torch.randn(*shape, generator=gen).to(torch.bfloat16).cuda()

    T, Hq, G, k = 1024, 8, 2, 4
    shape = msa.Shape(B=1, T=T, Hq=Hq, G=G, k=k)
    Q, K, V, dO = normal(1, T, Hq, 128), normal(1, T, G, 128), normal(1, T, G, 128), normal(1, T, Hq, 128)
    qi, ki = normal(1, T, G, 64), normal(1, T, 64)

    def run(stream=None):
        bi = msa.index_topk(shape, qi, ki, stream=stream)
        O, LSE = msa.sparse_fwd(shape, Q, K, V, bi, stream=stream)
        g = msa.bwd(shape, Q, K, V, O, dO, LSE, qi, ki, bi, stream=stream)
        Od, LSEd = msa.dense_fwd(shape, Q, K, V, stream=stream)
        gd = msa.dense_bwd(shape, Q, K, V, Od, dO, LSEd, qi, ki, stream=stream)
        return [bi, O, LSE, Od, LSEd, *g.values()], list(gd.values())

    same, near = ([x.clone() for x in part] for part in run())
    sizes = [x.nbytes for x in same + near] + [msa.msa_workspace_size(shape, w) for w in
                                        (msa.MSA_WS_TOPK, msa.MSA_WS_FWD, msa.MSA_WS_BWD, msa.MSA_WS_DENSE)]
    side, here = torch.cuda.Stream(), torch.cuda.current_stream()
    torch.cuda.synchronize()
    for _ in range(5):
        torch.cuda._sleep(3_000_000)
        for n in sizes:
            torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255)
        with torch.cuda.stream(side):
            torch.cuda._sleep(1_000_000)
        got = run(side.cuda_stream if raw else side)
        held = [torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255) for n in sizes]
        here.wait_stream(side)
        for a, b in zip(got[0], same):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        # msa_dense_bwd's sums come in another order from run to run (2^-24 a term); what another stream wrote is NaN here
        for a, b in zip(got[1], near):
            assert float((a - b).abs().max()) <= 2.0 ** -8 * float(b.abs().max())
        del got, held


def test_a_stream_of_another_device_is_refused(msa):
    import torch

    class Other:
        device = torch.device("cuda", 1)
        cuda_stream = 0

    q, k = torch.zeros(1, 128, 1, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, 128, 64, dtype=torch.bfloat16,
                                                                                        device="cuda")
    with pytest.raises(ValueError, match="cuda:1"):
        msa.index_topk(msa.Shape(B=1, T=128, Hq=1, G=1, k=1), q, k, stream=Other())
