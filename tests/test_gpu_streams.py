"""Calls on a stream that is not the current one: what the binding allocates for
them comes from the launching stream's pool, so nothing still queued on the
current stream can use the same memory."""
import pytest
import torch

import paged_gqa_decode_07_b200 as pgd
from tests.test_gpu_prefill import bits, cu_of, make_pages, randn

pytestmark = pytest.mark.gpu

HQ, HKV, D, BS = 8, 2, 128, 16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    pgd.load_library()
    yield
    assert pgd.get_device_error() == 0


def pool_of(t):
    """The stream handle whose pool holds a tensor's memory."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("the tensor is in no segment of the allocator")


def prompts(n, seed):
    return [randn((n, h, D), seed + i) for i, h in enumerate((HQ, HKV, HKV))]


@pytest.mark.parametrize("how", ["Stream", "handle"])
def test_memory_made_inside_a_call_is_the_launching_streams(how):
    """Prepared only: nothing is launched."""
    s = torch.cuda.Stream()
    stream = s if how == "Stream" else s.cuda_stream
    q, k, v = prompts(900, 1)
    cu_t = cu_of([900])[1]
    calls = [pgd.prefill_attention(q, k, v, cu_t, HQ, HKV, D, 0.09, num_ctas=3, stream=stream,
                                   prepare=True)]
    kc, vc, table, _, _ = make_pages([900], HKV, D, BS, "bf16", 4)
    ctx = torch.tensor([900], dtype=torch.int32, device="cuda")
    calls.append(pgd.paged_prefill_attention(q, kc, vc, table, ctx, cu_t, HQ, HKV, D, BS, 0.09,
                                             num_ctas=3, stream=stream, prepare=True))
    for c in calls:
        assert c._keep is not None and pool_of(c._keep) == s.cuda_stream
    one = q[:1].contiguous()
    calls += [
        pgd.kv_quant_scales(k, v, stream=stream, prepare=True),
        pgd.kv_gather(kc, vc, torch.arange(5, device="cuda"), stream=stream, prepare=True),
        pgd.paged_decode_attention(one, kc, vc, table, ctx, HQ, HKV, D, BS, 0.09, stream=stream,
                                   prepare=True),
        pgd.paged_decode_attention_ex(one[:, None], kc, vc, table, ctx, HQ, HKV, D, BS, 0.09,
                                      stream=stream, prepare=True),
        pgd.paged_decode_partial(one, kc, vc, table, ctx, HQ, HKV, D, BS, 0.09, stream=stream,
                                 prepare=True),
        pgd.decode_step(one, k[:1].contiguous(), v[:1].contiguous(), kc, vc, table, ctx, HQ, HKV,
                        D, BS, 0.09, stream=stream, prepare=True),
        pgd.merge_partials(torch.zeros((2, 3, D), device="cuda"),
                           torch.zeros((2, 3), device="cuda"), stream=stream, prepare=True)]
    for c in calls:
        for t in c.result if isinstance(c.result, tuple) else (c.result,):
            assert pool_of(t) == s.cuda_stream, c._name


def test_the_default_streams_handle_names_the_default_stream():
    q, k, v = prompts(900, 2)
    other = torch.cuda.Stream()
    with torch.cuda.stream(other):
        call = pgd.prefill_attention(q, k, v, cu_of([900])[1], HQ, HKV, D, 0.09, num_ctas=3,
                                     stream=0, prepare=True)
    assert pool_of(call._keep) == 0 and pool_of(call.result) == 0


def test_calls_on_the_current_and_on_another_stream_at_once():
    """Cut calls in turn on two streams that do not wait for one another."""
    n = 1500
    cu_t = cu_of([n])[1]
    data = [prompts(n, 10), prompts(n, 20)]
    want = [pgd.prefill_attention(*x, cu_t, HQ, HKV, D, 0.09, num_ctas=9).clone() for x in data]
    outs = [[torch.zeros_like(w) for w in want] for _ in range(20)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for o in outs:
        pgd.prefill_attention(*data[0], cu_t, HQ, HKV, D, 0.09, o[0], num_ctas=9)
        pgd.prefill_attention(*data[1], cu_t, HQ, HKV, D, 0.09, o[1], num_ctas=9, stream=s)
    torch.cuda.synchronize()
    for o in outs:
        for got, w in zip(o, want):
            assert torch.equal(bits(got), bits(w))


def test_an_output_made_on_another_stream_outlives_its_reader():
    """Freed while the current stream still reads it: the block is not handed
    to the other stream's next call before that."""
    n = 700
    cu_t = cu_of([n])[1]
    a, b = prompts(n, 30), prompts(n, 40)
    want = pgd.prefill_attention(*a, cu_t, HQ, HKV, D, 0.09).clone()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = pgd.prefill_attention(*a, cu_t, HQ, HKV, D, 0.09, stream=s)
    at = out.data_ptr()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(50_000_000)
    got = out.clone()
    del out
    after = pgd.prefill_attention(*b, cu_t, HQ, HKV, D, 0.09, stream=s)
    assert after.data_ptr() != at
    torch.cuda.synchronize()
    assert torch.equal(bits(got), bits(want))


@pytest.mark.parametrize("side", [False, True], ids=["captured", "joined"])
def test_a_captured_call_that_names_its_stream(side):
    """The capturing stream itself, or one that the capture forks to and joins;
    the output and the workspace are made inside the call."""
    n = 1500
    cu_t = cu_of([n])[1]
    q, k, v = prompts(n, 50)
    pgd.prefill_attention(q, k, v, cu_t, HQ, HKV, D, 0.09, num_ctas=9)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cur = torch.cuda.current_stream()
        on = s if side else cur
        if side:
            s.wait_stream(cur)
        out = pgd.prefill_attention(q, k, v, cu_t, HQ, HKV, D, 0.09, num_ctas=9, stream=on)
        if side:
            cur.wait_stream(s)
    for seed in (60, 70):
        for t, x in zip((q, k, v), prompts(n, seed)):
            t.copy_(x)
        g.replay()
        want = pgd.prefill_attention(q, k, v, cu_t, HQ, HKV, D, 0.09, num_ctas=9)
        torch.cuda.synchronize()
        assert torch.equal(bits(out), bits(want))
