"""Calls whose inputs the call before has just written (marked gpu): every launch is a
programmatic dependent of the one before it on the stream, so a kernel may read nothing until that
one is complete.  Each round writes other values over the same buffers, so a read ahead of the wait
finds the last round's; results are compared with the same calls after a synchronisation, bit by
bit, and those with the formula."""
import pytest
import torch

from test_gpu_linear import compare

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_31_gb300 as m
    m.load_library()
    return m


def rounds(run, inputs, draws, captured):
    """run(*buffers) in rounds, eagerly or replayed from a graph: the outputs of each round."""
    buffers = [t.clone() for t in inputs]
    outs = run(*buffers)
    torch.cuda.synchronize()
    graph = None
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = run(*buffers)
    results = []
    for values in draws:
        for b, v in zip(buffers, values):
            b.copy_(v)
        if graph is not None:
            graph.replay()
        else:
            outs = run(*buffers)
        results.append([o.clone() for o in outs])
    torch.cuda.synchronize()
    return results


@pytest.mark.parametrize("captured", [False, True], ids=["eager", "captured"])
@pytest.mark.parametrize("rows", [1, 2, 4, 40])
@pytest.mark.parametrize("N,K", [(1024, 4096), (130, 16384)])
def test_weight_written_by_the_call_before(sv, N, K, rows, captured):
    """out = x W^T with W = A B^T from the call before (keys from a projection, say)."""
    g = torch.Generator(device="cuda").manual_seed(rows + N)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)
    draws = [(rand(N, 512), rand(rows, K)) for _ in range(4)]
    b = rand(K, 512) * 0.05
    w = torch.empty(N, K, dtype=BF, device="cuda")
    out = torch.empty(rows, N, dtype=BF, device="cuda")

    def run(a, x):
        sv.spec_linear(a, b, out=w)
        sv.spec_linear(x, w, out=out)
        return out, w

    for (a, x), (got, w_got) in zip(draws, rounds(run, draws[0], draws, captured)):
        assert torch.equal(w_got, sv.spec_linear(a, b))
        torch.cuda.synchronize()
        assert torch.equal(got, sv.spec_linear(x, w_got))
        compare(got, x, w_got)
    assert sv.spec_verify_check() == sv.SPEC_OK


@pytest.mark.parametrize("B", [1, 12])
def test_logits_written_by_the_call_before(sv, B):
    """The verifies from logits, whose streaming pass loads the same way, behind the linear layer."""
    gamma, d, V = 3, 256, 8000
    g = torch.Generator(device="cuda").manual_seed(B)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)
    draws = [(rand(B, gamma + 1, d), rand(B, gamma, d)) for _ in range(4)]
    head = rand(V, d) * 0.2
    toks = torch.randint(0, V, (B, gamma), generator=g, device="cuda", dtype=torch.int32)
    lt = torch.empty(B, gamma + 1, V, dtype=BF, device="cuda")
    ld = torch.empty(B, gamma, V, dtype=BF, device="cuda")

    def run(ht, hd):
        sv.spec_linear(hd, head, out=ld)
        sv.spec_linear(ht, head, out=lt)
        t, n = sv.spec_verify_ex(lt, ld, toks, 1.0, 0.7, 3)[:2]
        sv.spec_linear(ht, head, out=lt)
        gt, gn = sv.spec_verify_greedy(lt, toks)[:2]
        return t, n, gt, gn

    for (ht, hd), got in zip(draws, rounds(run, draws[0], draws, False)):
        a, b = sv.spec_linear(ht, head), sv.spec_linear(hd, head)
        torch.cuda.synchronize()
        want = [*sv.spec_verify_ex(a, b, toks, 1.0, 0.7, 3)[:2], *sv.spec_verify_greedy(a, toks)[:2]]
        assert all(torch.equal(x, y) for x, y in zip(got, want))
