"""Calls with `stream=` name another stream than the caller's: what the call makes may not lie in
memory that either stream still uses.

Both streams are held up by a bounded sleep kernel, so that what is enqueued behind it has not run
when the next call is made; contents and addresses are looked at after both are idle.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
SLEEP = 40_000_000  # cycles, about 20 ms


def calls():
    from bit_moe_expert_route_gb300 import ops
    g = torch.Generator(device="cuda").manual_seed(0)

    def n(*shape):
        return torch.randn(*shape, generator=g, device="cuda").bfloat16()
    x, r, w = n(1024, 2048), n(1024, 2048), n(2048)
    a = torch.randint(-127, 128, (300, 1024), generator=g, device="cuda").to(torch.int8)
    b = torch.randint(-127, 128, (20000, 1024), generator=g, device="cuda").to(torch.int8)
    sa, sb = torch.rand(300, generator=g, device="cuda"), torch.rand(20000, generator=g, device="cuda")
    q, k, v = n(64, 16, 128), n(3000, 2, 128), n(3000, 2, 128)
    z, ids = n(40, 50000), torch.arange(40, dtype=torch.int32, device="cuda")
    gate = torch.rand(64, 2, generator=g, device="cuda")
    kg, vg, states = n(64, 1, 128), n(64, 2, 128), [torch.zeros(2, 128, 128, device="cuda") for _ in range(2)]
    logits = z[:, :256].float()
    return {
        "norm": lambda **o: ops.add_rmsnorm_q8(x, w, residual=r, values=True, **o),
        "product": lambda **o: ops.gemm_w8a8(a, sa, b, sb, **o),
        "attention": lambda **o: ops.prefix_attention(q, k, v, **o),
        "logprobs": lambda **o: ops.token_logprobs(z, ids, top_k=20, **o),
        "decode_attention": lambda **o: ops.decode_attention(q[0], k, v, **o),
        "scan": lambda **o: ops.gdn_scan(kg, kg, vg, gate, gate, states.pop(), **o),
        "route": lambda **o: ops.route(logits, 8, 64, **o),
    }


NAMES = ["norm", "product", "attention", "logprobs", "decode_attention", "scan", "route"]


def tensors(x):
    from bit_moe_expert_route_gb300 import ops
    return [t for t in ops._tensors(x) if t.numel()]


def span(t):
    return t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()


@pytest.mark.parametrize("name", NAMES)
def test_memory_in_use_on_the_callers_stream_is_not_taken(name):
    call = calls()[name]
    want = call()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    # blocks of the sizes that the call asks for, freed while the caller's stream has still to read them
    sizes = [t.numel() * t.element_size() for t in tensors(want)] + [256 << i for i in range(17)]
    blocks = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes]
    copies = [torch.empty_like(b) for b in blocks]
    torch.cuda.synchronize()
    torch.cuda._sleep(SLEEP)
    for b, c in zip(blocks, copies):
        c.copy_(b)
    spans = [span(b) for b in blocks]
    del blocks, b
    got = call(stream=s)
    taken = [(span(t), f) for t in tensors(got) for f in spans if span(t)[0] < f[1] and f[0] < span(t)[1]]
    torch.cuda.synchronize()
    assert not taken
    assert all(bool((c == 7).all()) for c in copies)
    for t, u in zip(tensors(got), tensors(want)):
        if name != "route" or t.shape == u.shape and t.is_floating_point():
            assert torch.equal(t, u)


@pytest.mark.parametrize("name", NAMES)
def test_results_are_kept_for_the_callers_stream(name):
    call = calls()[name]
    want = [t.clone() for t in tensors(call())]
    s, here = torch.cuda.Stream(), torch.cuda.current_stream()
    torch.cuda.synchronize()
    got = call(stream=s)
    here.wait_stream(s)
    torch.cuda._sleep(SLEEP)
    copies = [t.clone() for t in tensors(got)]
    sizes = [t.numel() * t.element_size() for t in tensors(got)]
    del got
    with torch.cuda.stream(s):
        for n in sizes * 2:
            torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    if name != "route":
        assert all(torch.equal(c, u) for c, u in zip(copies, want))
    else:
        assert torch.equal(copies[1], want[1])


def test_the_callers_own_stream():
    """Naming the current stream is the same as naming none."""
    for name, call in calls().items():
        if name != "route":
            a, b = tensors(call()), tensors(call(stream=torch.cuda.current_stream()))
            torch.cuda.synchronize()
            assert all(torch.equal(t, u) for t, u in zip(a, b)), name
