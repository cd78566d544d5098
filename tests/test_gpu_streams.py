"""Calls on another stream than the current one (stream=), while the two are at
work at different times: memory that one of them still uses is not given to
the other."""
import pytest

import test_gpu_logprob as logprob

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

N, VOCAB = 4096, 1500
BUSY = 400_000_000   # cycles, some 0.2 s


@pytest.fixture(scope="module")
def sq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import parity_binade_chunked_gb300 as sq
    return sq


@pytest.fixture(scope="module")
def inputs(sq):
    x, t, a = logprob.make(N, VOCAB, torch.bfloat16, 31)
    u = torch.rand(N, device="cuda")
    lses = sq.token_logprob(x, t)[1]
    return dict(x=x, t=t, a=a, u=u, lses=lses, list=sq.TensorList([x[:7], x[7:30]]))


def calls(sq, i):
    """Each call's name, and its results as a tuple, on a stream."""
    return {
        "sample": lambda s: sq.sample_tokens(i["x"], i["u"], top_k=50, top_p=0.9, stream=s),
        "logprob": lambda s: sq.token_logprob(i["x"], i["t"], stream=s),
        "grad": lambda s: sq.token_logprob_grad(i["x"], i["t"], i["a"], stream=s),
        "backward": lambda s: (sq.token_logprob_backward(i["x"], i["t"], i["a"], i["lses"], stream=s),),
        "norm": lambda s: (i["list"].norm(stream=s),),
    }


NAMES = ["sample", "logprob", "grad", "backward", "norm"]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("handle", [False, True])
def test_results_beside_a_busy_current_stream(sq, inputs, name, handle):
    """What the current stream has yet to write into memory that the host already freed does not land in results."""
    call = calls(sq, inputs)[name]
    want = call(None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    old = [torch.empty_like(w) for w in want]
    torch.cuda._sleep(BUSY)
    for o in old:
        o.fill_(7)
    del o, old   # given back while the current stream still has to write it
    got = call(side.cuda_stream if handle else side)
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(got, want))


def test_results_are_the_current_streams_to_free(sq, inputs):
    """A result freed while the current stream still reads it is not written by the other stream's next call."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    want, _ = sq.token_logprob(inputs["x"], inputs["t"])
    torch.cuda.synchronize()
    logps, lses = sq.token_logprob(inputs["x"], inputs["t"], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(BUSY)
    kept = logps.clone()
    del logps, lses
    for _ in range(4):
        sq.token_logprob(inputs["x"].neg(), inputs["t"], stream=side)
    torch.cuda.synchronize()
    assert torch.equal(kept, want)


def test_the_default_streams_handle(sq, inputs):
    side = torch.cuda.Stream()
    want, _ = sq.token_logprob(inputs["x"], inputs["t"])
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got, _ = sq.token_logprob(inputs["x"], inputs["t"], stream=0)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("name", NAMES[:-1])   # (a list keeps its tensors by itself)
@pytest.mark.parametrize("handle", [False, True])
def test_inputs_of_a_busy_stream(sq, inputs, name, handle):
    """Inputs given back, and their memory filled anew, before the other stream comes to the call."""
    want = calls(sq, inputs)[name](None)
    n = N
    side = torch.cuda.Stream()
    i = {k: v.clone() for k, v in inputs.items() if k != "list"}
    each = dict(temperature=torch.ones(n, device="cuda"), top_k=torch.full((n,), 50, device="cuda", dtype=torch.int32),
                top_p=torch.full((n,), 0.9, device="cuda"), min_p=torch.zeros(n, device="cuda"))
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    s = side.cuda_stream if handle else side
    if name == "sample":
        got = sq.sample_tokens(i["x"], i["u"], stream=s, **each)
    else:
        got = calls(sq, i)[name](s)
    shapes = [(t.shape, t.dtype) for d in (i, each) for t in d.values()]
    i.clear()
    each.clear()
    filled = [torch.full(shape, 0.5 if dtype.is_floating_point else 1, device="cuda", dtype=dtype)
              for shape, dtype in shapes for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(got, want)) and filled


def test_a_given_result_of_a_busy_stream(sq, inputs):
    """A result's memory given back before the other stream has written it is not another tensor's when it does."""
    side = torch.cuda.Stream()
    logps, lses = torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    sq.token_logprob(inputs["x"], inputs["t"], logps=logps, lses=lses, stream=side)
    del logps, lses
    filled = [torch.full((N,), 0.5, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert all((f == 0.5).all() for f in filled)
