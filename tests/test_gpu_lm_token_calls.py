"""GPU: what calls of the operators beside the 8-bit ones leave to their caller and what they do not: both
ways of the binding, given streams, captured calls, several calls at once, threads."""
from __future__ import annotations

import threading
import time

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only machines, never run there
    pytest.skip("no CUDA device", allow_module_level=True)

from dac_vocoder_decode_gb300 import binding as V  # noqa: E402
from tests import test_gpu_lm_token as T  # noqa: E402

SYNC = V.VOC_FLAG_SYNC


def _calls(seed=0, rows=64):
    """A call of each operator: (call, inputs that a second set may replace in place)."""
    g = T._gen(seed)
    q, k = T._randn(g, rows, 6, 64).bfloat16(), T._randn(g, rows, 2, 64).bfloat16()
    w = (1 + 0.1 * T._randn(g, 64)).bfloat16()
    pos = torch.randint(0, 9999, (rows,), generator=g, device="cuda", dtype=torch.int32)
    turns = V.rotation_turns(T._rates(32))
    c = T.Adapters(rows, 320, 256, 16, 5, "bf16", seed=seed)
    x = T._randn(g, rows, 5003)
    tokens = torch.randint(0, 5003, (rows,), generator=g, device="cuda")
    return {
        "rotate": (lambda **kw: V.rotate_heads(q, k, pos, turns, q_weight=w, k_weight=w, **kw), (q, k, pos)),
        "adapters": (lambda **kw: (V.adapters_fp8(c.y, c.x, c.x_scale, c.a, c.b, c.scale, c.ids, **kw),),
                     (c.y, c.x8, c.x_scale, c.ids)),
        "logprobs": (lambda **kw: V.logprobs(x, tokens, top=7, temperature=0.8, **kw), (x, tokens))}


OPS = ["rotate", "adapters", "logprobs"]


def _same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("op", OPS)
def test_both_ways_of_the_binding(op, monkeypatch):
    call, _ = _calls()[op]
    a = call(flags=SYNC)
    monkeypatch.setattr(V._LM, "fast", None)
    b = call(flags=SYNC)
    assert _same(a, b) and [t.dtype for t in a] == [t.dtype for t in b]


@pytest.mark.parametrize("fast", [True, False])
def test_both_ways_refuse_alike(fast, monkeypatch):
    if not V._LM.ready:
        V._lm_setup()
    if not fast:
        monkeypatch.setattr(V._LM, "fast", None)
    q = torch.zeros(4, 2, 64, device="cuda").half()
    pos, turns = torch.zeros(4, dtype=torch.int32, device="cuda"), V.rotation_turns(T._rates(32))
    c = T.Adapters(4, 16, 32, 8, 2)
    x, tok = torch.zeros(4, 8, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    bad = [lambda: V.rotate_heads(q[:, :, :60], None, pos, turns), lambda: V.rotate_heads(q, q[:3], pos, turns),
           lambda: V.rotate_heads(q, None, pos[:3], turns), lambda: V.rotate_heads(q, None, pos.long(), turns),
           lambda: V.rotate_heads(q, None, pos, turns[1:]), lambda: V.rotate_heads(q, None, pos, turns.double()),
           lambda: V.rotate_heads(q, None, pos, turns, k_weight=q[0, 0]),
           lambda: V.rotate_heads(q, None, pos, turns, q_weight=q[0, 0].bfloat16()),
           lambda: V.rotate_heads(q, q, pos, turns, k_out=q[:, :1]),
           lambda: V.rotate_heads(q.transpose(1, 2), None, pos, turns),
           lambda: V.rotate_heads(q, None, pos, turns, axis=pos),
           lambda: c.run(y=c.y[:3]), lambda: c.run(y=c.y.half()), lambda: c.run(out=c.y.float()),
           lambda: V.adapters_fp8(c.y, c.x, c.x_scale, c.a, c.b[:1], c.scale, c.ids),
           lambda: V.adapters_fp8(c.y, c.x, c.x_scale, c.a, c.b, c.scale, c.ids.long()),
           lambda: V.adapters_fp8(c.y, c.x, c.x_scale, c.a[:, :4].contiguous(), c.b[:, :, :4], c.scale, c.ids),
           lambda: V.adapters_fp8(c.y, c.x, c.x_scale[:2], c.a, c.b, c.scale, c.ids),
           lambda: V.logprobs(x, tok.int()), lambda: V.logprobs(x, tok[:2]), lambda: V.logprobs(x, top=9),
           lambda: V.logprobs(x, top=-1), lambda: V.logprobs(x.T), lambda: V.logprobs(x, temperature=0.0),
           lambda: V.logprobs(torch.zeros(2, 100, device="cuda"), top=33)]
    for i, call in enumerate(bad):
        with pytest.raises(V.VocoderError) as e:
            call()
        assert e.value.status in (V.VOC_INVALID_ARG, V.VOC_UNSUPPORTED), i


@pytest.mark.parametrize("op", OPS)
def test_captured_calls_take_the_inputs_of_the_replay(op):
    call, inputs = _calls(1)[op]
    fresh, other = _calls(2)[op]
    want = fresh(flags=SYNC)
    call(flags=SYNC)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        first = call()
        second = call()
    for a, b in zip(inputs, other):
        a.copy_(b)
    if op == "adapters":  # the pools of the second set differ: its result on the first one's pools
        want = call(flags=SYNC)
    graph.replay()
    torch.cuda.synchronize()
    assert _same(first, second)
    assert op == "rotate" or _same(first, want)
    if op == "rotate":  # the weights of the second set differ too
        assert _same(first, call(flags=SYNC))


@pytest.mark.parametrize("op", OPS)
def test_given_stream(op):
    """On another stream: the result is there once that stream is done, and memory that the current stream
    still reads is left alone."""
    call, _ = _calls(3)[op]
    want = [t.clone() for t in call(flags=SYNC)]
    side = torch.cuda.Stream()
    got = call(stream=side)
    side.synchronize()
    assert _same(got, want)
    size = sum(t.numel() * t.element_size() for t in want[:1])
    torch.cuda.synchronize()
    del got
    torch.cuda.empty_cache()
    old = torch.full((size,), 77, dtype=torch.uint8, device="cuda")
    kept = torch.empty_like(old)
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)  # about 0.2 s
    kept.copy_(old)
    del old
    got = call(stream=side)
    torch.cuda.synchronize()
    assert bool((kept == 77).all()) and _same(got, want)


@pytest.mark.parametrize("op", OPS)
def test_two_streams_at_once(op):
    (a, _), (b, _) = _calls(4)[op], _calls(5, rows=300)[op]
    want_a, want_b = a(flags=SYNC), b(flags=SYNC)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(20):
        got.append((a(), b(stream=side)))
    torch.cuda.synchronize()
    assert all(_same(x, want_a) and _same(y, want_b) for x, y in got)


@pytest.mark.parametrize("op", OPS)
def test_inputs_made_just_before(op):
    """Inputs that the kernel in front of the call writes."""
    call, inputs = _calls(6)[op]
    others = [[t.clone() for t in _calls(7 + i)[op][1]] for i in range(8)]
    got = []
    for set_ in others:
        for a, b in zip(inputs, set_):
            a.copy_(b)
        got.append(call())
    torch.cuda.synchronize()
    for set_, g in zip(others, got):
        for a, b in zip(inputs, set_):
            a.copy_(b)
        torch.cuda.synchronize()
        assert _same(g, call(flags=SYNC))


@pytest.mark.parametrize("op", OPS)
def test_other_threads_run_while_a_call_waits_for_its_stream(op):
    call, _ = _calls(8)[op]
    call()
    waited = []

    def wait():
        torch.cuda._sleep(1_000_000_000)
        start = time.perf_counter()
        call(flags=SYNC)
        waited.append(time.perf_counter() - start)

    thread = threading.Thread(target=wait)
    thread.start()
    last, gap = time.perf_counter(), 0.0
    while thread.is_alive():
        time.sleep(0.005)
        now = time.perf_counter()
        gap, last = max(gap, now - last), now
    thread.join()
    assert waited and waited[0] > 0.25
    assert gap < 0.2


def test_more_tokens_than_32_bits_of_bytes():
    """Offsets beyond 2^31 elements: the last rows of large tensors."""
    rows, vocab = 70000, 33000  # 2.3e9 logits, bf16
    x = torch.zeros(rows, vocab, dtype=torch.bfloat16, device="cuda")
    g = T._gen(1)
    x[-300:] = (T._randn(g, 300, vocab) * 3).bfloat16()
    tokens = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    got = V.logprobs(x, tokens, top=3, flags=SYNC)
    T._check_logprobs(x[-300:], tokens[-300:], 3, 1.0, [t[-300:] for t in got])
    del x
    tokens, heads = 300000, 60  # 2.3e9 values of q
    q = torch.zeros(tokens, heads, 128, dtype=torch.bfloat16, device="cuda")
    q[-50:] = T._randn(g, 50, heads, 128).bfloat16()
    pos = torch.arange(tokens, dtype=torch.int32, device="cuda")
    rates = T._rates(64)
    V.rotate_heads(q[:-50], None, pos[:-50], V.rotation_turns(rates), q_out=q[:-50], flags=SYNC)
    want = V.rotate_heads(q[-50:].clone(), None, pos[-50:].clone(), V.rotation_turns(rates), flags=SYNC)[0]
    V.rotate_heads(q, None, pos, V.rotation_turns(rates), q_out=q, flags=SYNC)
    assert torch.equal(q[-50:], want)
    del q
    M, N = 150000, 16000  # 2.4e9 outputs
    c = T.Adapters(200, N, 64, 8, 2)
    y = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    y[-200:] = c.y
    x = torch.zeros(M, 64, dtype=torch.uint8, device="cuda")
    x[-200:] = c.x8
    xs, ids = torch.ones(M, device="cuda"), torch.full((M,), -1, dtype=torch.int32, device="cuda")
    xs[-200:], ids[-200:] = c.x_scale, c.ids
    V.adapters_fp8(y, x.view(torch.float8_e4m3fn), xs, c.a, c.b, c.scale, ids, out=y, flags=SYNC)
    c.check(y[-200:])
    assert not bool(y[:1000].any())
